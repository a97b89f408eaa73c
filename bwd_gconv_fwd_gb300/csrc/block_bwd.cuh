// block_bwd.cuh -- the block norm / join backward kernels' instances and launches.
#include "block_internal.h"
#include "block_row.cuh"
#include "block_stage.cuh"

namespace gconv {

namespace {

template <void (*Kernel)(BlockArgs, StageMaps)>
void launch_staged(const BlockShape &s, const BlockArgs &a, const StageMaps &maps, cudaStream_t st)
{
    static bool attr[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return;   // the error stays for the caller's check
    if (!attr[dev]) {
        if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBlockSmem) != cudaSuccess) return;
        attr[dev] = true;
    }
    launch_dependent_clusters(Kernel, s.grid, s.threads, s.smem, s.cluster, st, a, maps);
}

template <typename T, int VEC>
void staged(int kind, const BlockShape &s, const BlockArgs &a, const StageMaps &maps, cudaStream_t st)
{
    const int gate = a.gate != GCONV_GATE_FULL ? kGateOff : a.act == GCONV_ACT_SILU ? kGateSilu : kGateOther;
    if (kind == kBlockNorm) launch_staged<block_bwd_stage_kernel<T, VEC, false, true, kGateOff>>(s, a, maps, st);
    else if (kind == kBlockJoin && gate == kGateOff) launch_staged<block_bwd_stage_kernel<T, VEC, true, false, kGateOff>>(s, a, maps, st);
    else if (kind == kBlockJoin && gate == kGateSilu) launch_staged<block_bwd_stage_kernel<T, VEC, true, false, kGateSilu>>(s, a, maps, st);
    else if (kind == kBlockJoin) launch_staged<block_bwd_stage_kernel<T, VEC, true, false, kGateOther>>(s, a, maps, st);
    else if (gate == kGateOff) launch_staged<block_bwd_stage_kernel<T, VEC, true, true, kGateOff>>(s, a, maps, st);
    else if (gate == kGateSilu) launch_staged<block_bwd_stage_kernel<T, VEC, true, true, kGateSilu>>(s, a, maps, st);
    else launch_staged<block_bwd_stage_kernel<T, VEC, true, true, kGateOther>>(s, a, maps, st);
}

template <typename T, int VEC, int NV>
void rows(int kind, const BlockShape &s, const BlockArgs &a, cudaStream_t st)
{
    if (kind == kBlockNorm) launch_dependent(block_bwd_row_kernel<T, VEC, NV, false, true>, s.grid, s.threads, s.smem, st, a);
    else if (kind == kBlockJoin) launch_dependent(block_bwd_row_kernel<T, VEC, NV, true, false>, s.grid, s.threads, s.smem, st, a);
    else launch_dependent(block_bwd_row_kernel<T, VEC, NV, true, true>, s.grid, s.threads, s.smem, st, a);
}

template <typename T>
void launch_t(int kind, const BlockShape &s, const BlockArgs &a, const StageMaps &maps, cudaStream_t st)
{
    if (s.row) {
        constexpr int V = 16 / (int)sizeof(T);
        if (s.vec == 1) rows<T, 1, kRowHeld>(kind, s, a, st);
        else if (s.held == kRowHeld) rows<T, V, kRowHeld / V>(kind, s, a, st);
        else rows<T, V, 2 * kRowHeld / V>(kind, s, a, st);
    } else if (s.staged) {
        if (s.vec == 1) staged<T, 1>(kind, s, a, maps, st);
        else if (s.vec == 2) staged<T, 2>(kind, s, a, maps, st);
        else if (s.vec == 4) staged<T, 4>(kind, s, a, maps, st);
        else if constexpr (sizeof(T) == 2) staged<T, 8>(kind, s, a, maps, st);
    } else if (kind == kBlockNorm)
        launch_dependent(block_bwd_walk_kernel<T, false, true>, s.grid, s.threads, s.smem, st, a);
    else if (kind == kBlockJoin)
        launch_dependent(block_bwd_walk_kernel<T, true, false>, s.grid, s.threads, s.smem, st, a);
    else
        launch_dependent(block_bwd_walk_kernel<T, true, true>, s.grid, s.threads, s.smem, st, a);
}

}  // namespace

}  // namespace gconv
