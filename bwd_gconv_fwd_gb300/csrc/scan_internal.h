// scan_internal.h -- what the selective scan's translation units share.
#pragma once

#include "scan.cuh"

namespace gconv {

// The shape of one launch (scan.cu, scan_shape).
struct ScanShape {
    int form;                 // kScanForms of the direction
    int warps, vec;
    unsigned grid;
    size_t smem;
};

// Time lanes, positions a thread and channels a thread of the forms.
struct ScanForm { int TL, K, P; };
constexpr ScanForm kFwdForms[] = {{8, 16, 2}, {8, 8, 2}, {8, 16, 1}, {32, 8, 1}, {32, 16, 1}};
constexpr ScanForm kBwdForms[] = {{8, 8, 2}, {8, 8, 1}};
constexpr int kFwdFormCount = sizeof(kFwdForms) / sizeof(kFwdForms[0]), kBwdFormCount = sizeof(kBwdForms) / sizeof(kBwdForms[0]);

void scan_fwd_bf16(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st);
void scan_fwd_f32(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st);
void scan_bwd_bf16(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st);
void scan_bwd_f32(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st);

}  // namespace gconv
