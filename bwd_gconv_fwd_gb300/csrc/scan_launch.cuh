// scan_launch.cuh -- picks the instance of a scan kernel that a shape names.
#pragma once

#include "scan_bwd.cuh"
#include "scan_ends.cuh"
#include "scan_fwd.cuh"
#include "scan_internal.h"

namespace gconv {

template <typename F>
void scan_start(F *kernel, const ScanShape &s, const ScanArgs &a, cudaStream_t st)
{
    if (s.smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s.smem) != cudaSuccess)
        return;
    launch_dependent(kernel, s.grid, (unsigned)s.warps * 32, s.smem, st, a);
}

template <typename T>
void scan_fwd_start(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st)
{
    if (s.vec) scan_start(ends ? scan_ends_kernel<T, true, false> : scan_fwd_kernel<T, true>, s, a, st);
    else scan_start(ends ? scan_ends_kernel<T, false, false> : scan_fwd_kernel<T, false>, s, a, st);
}

template <typename T, bool VEC>
void scan_bwd_pick(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st)
{
    if (ends) scan_start(scan_ends_kernel<T, VEC, true>, s, a, st);
    else if (!scan_keeps<T> && a.z) scan_start(scan_bwd_kernel<T, VEC, !scan_keeps<T>>, s, a, st);
    else scan_start(scan_bwd_kernel<T, VEC, false>, s, a, st);
}

template <typename T>
void scan_bwd_start(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st)
{
    if (s.vec) scan_bwd_pick<T, true>(s, ends, a, st);
    else scan_bwd_pick<T, false>(s, ends, a, st);
}

}  // namespace gconv
