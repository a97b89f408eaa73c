// scan_launch.cuh -- picks the instance of a scan kernel that a shape names.
#pragma once

#include "scan_bwd.cuh"
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

template <typename T, int F = 0>
void scan_fwd_start(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st)
{
    constexpr ScanForm f = kFwdForms[F];
    if (s.form == F) {
        if (s.vec) {
            if (ends) scan_start(scan_fwd_kernel<T, f.TL, f.K, f.P, true, true>, s, a, st);
            else scan_start(scan_fwd_kernel<T, f.TL, f.K, f.P, true, false>, s, a, st);
        } else {
            if (ends) scan_start(scan_fwd_kernel<T, f.TL, f.K, f.P, false, true>, s, a, st);
            else scan_start(scan_fwd_kernel<T, f.TL, f.K, f.P, false, false>, s, a, st);
        }
        return;
    }
    if constexpr (F + 1 < kFwdFormCount) scan_fwd_start<T, F + 1>(s, ends, a, st);
}

template <typename T, int F = 0>
void scan_bwd_start(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st)
{
    constexpr ScanForm f = kBwdForms[F];
    if (s.form == F) {
        if (s.vec) {
            if (ends) scan_start(scan_bwd_ends_kernel<T, f.TL, f.K, f.P, true>, s, a, st);
            else scan_start(scan_bwd_kernel<T, f.TL, f.K, f.P, true>, s, a, st);
        } else {
            if (ends) scan_start(scan_bwd_ends_kernel<T, f.TL, f.K, f.P, false>, s, a, st);
            else scan_start(scan_bwd_kernel<T, f.TL, f.K, f.P, false>, s, a, st);
        }
        return;
    }
    if constexpr (F + 1 < kBwdFormCount) scan_bwd_start<T, F + 1>(s, ends, a, st);
}

}  // namespace gconv
