// newton.cuh -- what the orthogonalisation's translation units share (newton.cu,
// newton_small.cu).
#pragma once

#include "internal.h"
#include "ptx.cuh"

#include <cuda_fp16.h>

namespace gconv {

constexpr float kNewtonScale = 256.f;   // 2^8, the scale of X, A and P in fp16

// The default coefficients: the quintic whose slope at zero is the largest that keeps every
// singular value within about 0.7 to 1.2 after five steps.
constexpr float kNewtonCoeffs[3] = {3.4445f, -4.7750f, 2.0315f};
constexpr int kNewtonSteps = 64;        // at most

// What the last product of a call writes.
struct NewtonOut {
    void *out;                   // orthogonalise: the result
    int out_bf16;
    const float *w;              // Muon: weights read and written
    float *w_out;
    __nv_bfloat16 *w_bf16;
    float keep, rate;            // w' = keep w - rate o
    int muon, tall;
};

// What the first kernels read.
struct NewtonIn {
    const void *g;
    int g_bf16;
    const float *m;              // Muon momentum, or nullptr
    float *m_out;
    float beta;
    int nesterov, tall;
    int64_t elems;               // of one matrix
    int rows, cols;              // of one matrix as it lies in memory
    float eps;
};

__device__ __forceinline__ float load_g(const NewtonIn &p, int64_t i)
{
    return p.g_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.g)[i]) : static_cast<const float *>(p.g)[i];
}

// The matrix that is orthogonalised, at one element: g, or the momentum's lookahead.  m is
// the updated momentum at the element.
__device__ __forceinline__ float lookahead(const NewtonIn &p, float g, float m)
{
    return p.nesterov ? fmaf(p.beta, m, g) : m;
}

// One element (at, in the caller's layout) of the result.
__device__ __forceinline__ void store_result(const NewtonOut &o, int64_t at, float v)
{
    if (o.muon) {
        v = fmaf(-o.rate, v, o.keep * o.w[at]);
        o.w_out[at] = v;
        if (o.w_bf16) o.w_bf16[at] = __float2bfloat16_rn(v);
    } else if (o.out_bf16) {
        static_cast<__nv_bfloat16 *>(o.out)[at] = __float2bfloat16_rn(v);
    } else {
        static_cast<float *>(o.out)[at] = v;
    }
}

// fp16 instruction descriptor: f16 A and B, f32 accumulator
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn_major)
{
    return (1u << 4) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The matrices of a call: m <= n, X is m x n.
struct NewtonShape {
    int G, rows, cols, m, n, tall, ldx, lda;
    size_t x_bytes, a_bytes, ws;
};

// Matrices whose shorter side fits one tile, in one launch each call (newton_small.cu).
bool newton_small_fits(const NewtonShape &s);
gconv_status newton_small_launch(const NewtonShape &s, const NewtonIn &in, const NewtonOut &out, int steps,
                                 const float *coeffs, unsigned int *err, cudaStream_t st);

}  // namespace gconv
