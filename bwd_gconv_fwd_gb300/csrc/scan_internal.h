// scan_internal.h -- what the selective scan's translation units share.
#pragma once

#include "scan.cuh"

namespace gconv {

// The shape of one launch (scan.cu, plan_scan).
struct ScanShape {
    int warps, vec;
    unsigned grid;
    size_t smem;
};

void scan_fwd_bf16(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st);
void scan_fwd_f32(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st);
void scan_bwd_bf16(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st);
void scan_bwd_f32(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st);

}  // namespace gconv
