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

template <typename T>
void scan_bwd_start(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st)
{
    if (s.vec) scan_start(ends ? scan_ends_kernel<T, true, true> : scan_bwd_kernel<T, true>, s, a, st);
    else scan_start(ends ? scan_ends_kernel<T, false, true> : scan_bwd_kernel<T, false>, s, a, st);
}

}  // namespace gconv
