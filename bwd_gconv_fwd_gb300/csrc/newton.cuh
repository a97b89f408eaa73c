// newton.cuh -- what the orthogonalisation's translation units share (newton.cu,
// newton_small.cu, newton_tiny.cu).
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

// scale / (|u| + eps) from the sum of squares; 0, so that zeros stay zeros, where that is infinite (a
// matrix of zeros, or whose squares are below fp32, without an eps).
__device__ __forceinline__ float unit_factor(float scale, float squares, float eps)
{
    const float f = scale / (sqrtf(squares) + eps);
    return isinf(f) ? 0.f : f;
}

// One element (at, in the caller's layout) of what a call writes: o, or the updated weight.
__device__ __forceinline__ void put_result(const NewtonOut &o, int64_t at, float v)
{
    if (o.muon) {
        o.w_out[at] = v;
        if (o.w_bf16) o.w_bf16[at] = __float2bfloat16_rn(v);
    } else if (o.out_bf16) {
        static_cast<__nv_bfloat16 *>(o.out)[at] = __float2bfloat16_rn(v);
    } else {
        static_cast<float *>(o.out)[at] = v;
    }
}

// The same from the orthogonalised matrix.
__device__ __forceinline__ void store_result(const NewtonOut &o, int64_t at, float v)
{
    put_result(o, at, o.muon ? fmaf(-o.rate, v, o.keep * o.w[at]) : v);
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Arrives at the barrier that stands at this block's offset `bar` in block `rank` of the cluster.
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar, uint32_t rank)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(ptx::map_to(bar, rank)) : "memory");
}

// A 3D tensor-map load into this block's shared memory that signals a barrier of its pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const void *tmap, int c0, int c1, int c2, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(bar) : "memory");
}

// Tensor memory of both blocks of a pair; one warp of each calls these.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
}

__device__ __forceinline__ void tmem_relinquish_pair()
{
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// The pair's product: 128 rows of D and A and half of B's columns in each block, at the same offsets.
__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

// Arrives at `bar` of both blocks once the products issued so far have ended.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(bar), "h"((uint16_t)3) : "memory");
}

// The same for `bar` of this block alone.
__device__ __forceinline__ void mma_commit_pair_here(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// fp16 instruction descriptor: f16 A and B, f32 accumulator
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn_major)
{
    return (1u << 4) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The matrices of a call: m <= n, X is m x n.
struct NewtonShape {
    int G, rows, cols, m, n, tall, ldx, lda, parts;
    size_t x_bytes, a_bytes, part_bytes, ws;
};

// Matrices of at most 16 x 1024 in fp32 (newton_tiny.cu).
bool newton_tiny_fits(const NewtonShape &s);
gconv_status newton_tiny_launch(const NewtonShape &s, const NewtonIn &in, const NewtonOut &out, int steps,
                                const float *coeffs, cudaStream_t st);

// Matrices whose shorter side fits one tile, in one launch each call (newton_small.cu).
bool newton_small_fits(const NewtonShape &s);
gconv_status newton_small_launch(const NewtonShape &s, const NewtonIn &in, const NewtonOut &out, int steps,
                                 const float *coeffs, unsigned int *err, cudaStream_t st);

}  // namespace gconv
