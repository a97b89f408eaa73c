// block_bwd.cu -- the block norm / join backward kernels' instances and launches.
#include "block_internal.h"

namespace gconv {

namespace {

template <typename T, int VEC, bool ONE>
void launch(int kind, const BlockShape &s, const BlockArgs &a, cudaStream_t st)
{
    constexpr int NCH = block_nch(VEC);
    if (kind == kBlockNorm)
        launch_dependent(block_bwd_kernel<T, VEC, NCH, false, true, ONE>, s.grid, s.threads, s.smem, st, a);
    else if (kind == kBlockJoin)
        launch_dependent(block_bwd_kernel<T, VEC, NCH, true, false, ONE>, s.grid, s.threads, s.smem, st, a);
    else
        launch_dependent(block_bwd_kernel<T, VEC, NCH, true, true, ONE>, s.grid, s.threads, s.smem, st, a);
}

template <typename T>
void launch_t(int kind, const BlockShape &s, const BlockArgs &a, cudaStream_t st)
{
    if (!s.one) launch<T, 1, false>(kind, s, a, st);
    else if (s.vec == 1) launch<T, 1, true>(kind, s, a, st);
    else if (s.vec == 2) launch<T, 2, true>(kind, s, a, st);
    else if (s.vec == 4) launch<T, 4, true>(kind, s, a, st);
    else if constexpr (sizeof(T) == 2) launch<T, 8, true>(kind, s, a, st);
}

}  // namespace

void block_bwd_launch(int kind, gconv_dtype dt, const BlockShape &s, const BlockArgs &a, cudaStream_t st)
{
    if (dt == GCONV_BF16) launch_t<__nv_bfloat16>(kind, s, a, st);
    else launch_t<float>(kind, s, a, st);
}

}  // namespace gconv
