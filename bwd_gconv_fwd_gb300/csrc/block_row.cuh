// block_row.cuh -- the block norm / join kernels for planes of one position (tokens, pooled
// features): an image's group is then Cg elements in a run, so the sums go along memory.
//
// TY threads hold a row, VEC neighbouring channels (16 bytes, or one where Cg is not a multiple) times
// NV each, in registers from the loads to the stores; Z rows a block, and blocks walk the rows.  Every
// tensor crosses the memory once, as 16-byte loads that are all in flight before the first
// sum.  The gradients' channel sums stay in registers until a block's last row (a block keeps to one
// group), so their partial sums are a block's and not an image's.
//
// Measured, [65536,1024] (the staged kernels' time, with their sums per image, in brackets): norm bf16
// 59 us, 4.5 TB/s (172), its gradient 142, 2.8 TB/s (1409); fp32 85, 6.3 TB/s (161), and 149, 5.4 TB/s
// (1388).  Join with next norm and a full silu gate, bf16 186, 3.6 TB/s (429), its gradient 465, 2.3 TB/s
// (3792); fp32 202, 6.6 TB/s (542), and 430, 5.0 TB/s (3754).  The memory is fp32's limit.  bf16, with twice the
// elements a byte, has none of its own: 19, 50, 72 and 133 instructions an element keep the issue slots 54, 61,
// 65 and 48 % busy at 38, 28, 29 and 16 warps an SM, which wait for their loads, as a block starts a row's
// only after the row before, and for their own results.  [8,1024] bf16, a launch: 1.9 us.
#pragma once

#include "block_norm.cuh"

namespace gconv {

constexpr int kRowThreads = 512;   // a row's, at most
constexpr int kRowHeld = 8;        // channels a thread holds, or twice that

// Adds v over the TY threads of a row, the same bits in each.  `red`: two halves of a float a warp and
// sum (`turn`: a half is written again two barriers after it was read).
template <int NS>
__device__ __forceinline__ void row_sum(float (&v)[NS], float *red, int TY, int &turn)
{
    #pragma unroll
    for (int q = 0; q < NS; ++q)
        for (int k = TY < 32 ? TY >> 1 : 16; k; k >>= 1) v[q] += __shfl_xor_sync(0xffffffffu, v[q], k);
    if (TY <= 32) return;
    const int warp = threadIdx.x >> 5, per = TY >> 5, all = blockDim.x >> 5;
    float *half = red + turn * NS * all;
    if ((threadIdx.x & 31) == 0)
        #pragma unroll
        for (int q = 0; q < NS; ++q) half[q * all + warp] = v[q];
    __syncthreads();
    const int first = warp / per * per;
    #pragma unroll
    for (int q = 0; q < NS; ++q) {
        v[q] = half[q * all + first];
        for (int k = 1; k < per; ++k) v[q] += half[q * all + first + k];
    }
    turn ^= 1;
}

// VEC elements from element `at`; zeros where there is no tensor or no channel.
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> row_load(const void *p, int64_t at, bool ok)
{
    Pack<T, VEC> v{};
    if (p && ok) v = *reinterpret_cast<const Pack<T, VEC> *>(static_cast<const T *>(p) + at);
    return v;
}

// VEC fp32 results: 16 bytes at a time, as the caller's pointers are aligned.
template <int VEC>
__device__ __forceinline__ void row_floats(float *p, const float (&v)[VEC])
{
    if constexpr (VEC >= 4) {
        #pragma unroll
        for (int k = 0; k < VEC; k += 4) *reinterpret_cast<float4 *>(p + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
    } else {
        p[0] = v[0];
    }
}

// VEC of a channel's fp32 numbers; ones where there are none.
template <int VEC>
__device__ __forceinline__ void row_weights(const float *p, int c, bool ok, float (&v)[VEC])
{
    #pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = 1.f;
    if (!p || !ok) return;
    if constexpr (VEC >= 4) {
        #pragma unroll
        for (int k = 0; k < VEC; k += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(p + c + k);
            v[k] = q.x; v[k + 1] = q.y; v[k + 2] = q.z; v[k + 3] = q.w;
        }
    } else {
        v[0] = p[c];
    }
}

template <int VEC>
__device__ __forceinline__ void branch_weights(const BlockArgs &a, int c, bool ok, float (&v)[VEC])
{
    float s[VEC];
    row_weights<VEC>(a.w, c, ok, v);
    row_weights<VEC>(a.s, c, ok, s);
    #pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = __fmul_rn(v[k], s[k]);
}

// Forward: three steps a row (sum h^2; out and sum out^2; next), a norm alone two.
template <typename T, int VEC, int NV, bool POST, bool NEXT>
__global__ void __launch_bounds__(kRowThreads) block_fwd_row_kernel(const BlockArgs a)
{
    __shared__ float red[2 * (kRowThreads / 32)];
    const int ty = threadIdx.x % a.TY, z = threadIdx.x / a.TY;
    int turn = 0;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    for (unsigned row0 = blockIdx.x * a.Z; row0 < (unsigned)a.rows; row0 += gridDim.x * a.Z) {
        const unsigned row = row0 + z;
        const int ch0 = row % (unsigned)a.G * a.Cg;
        const int64_t base = (int64_t)row * a.Cg;
        Pack<T, VEC> px[NV], ph[NV], pz[NV];
        bool ok[NV];
        #pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (ty + j * a.TY) * VEC;
            ok[j] = row < (unsigned)a.rows && c < a.Cg;
            px[j] = row_load<T, VEC>(a.x, base + c, ok[j]);
            if (POST) ph[j] = row_load<T, VEC>(a.h, base + c, ok[j]);
            if (POST) pz[j] = row_load<T, VEC>(a.z, base + c, ok[j]);
        }
        float o[NV][VEC], sum[1] = {0.f};
        #pragma unroll
        for (int j = 0; j < NV; ++j)
            #pragma unroll
            for (int k = 0; k < VEC; ++k) {
                o[j][k] = to_f(POST ? ph[j].v[k] : px[j].v[k]);
                sum[0] = fmaf(o[j][k], o[j][k], sum[0]);
            }
        row_sum<1>(sum, red, a.TY, turn);
        float r = rsqrtf(fmaf(sum[0], a.inv_cg, a.eps));
        if (POST) {
            sum[0] = 0.f;
            #pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (ty + j * a.TY) * VEC;
                float kc[VEC];
                branch_weights<VEC>(a, ch0 + c, ok[j], kc);
                #pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    if (a.gate != GCONV_GATE_NONE) kc[k] = __fmul_rn(kc[k], gate_value(to_f(pz[j].v[k]), a.act));
                    o[j][k] = fmaf(kc[k], __fmul_rn(o[j][k], r), to_f(px[j].v[k]));
                    sum[0] = fmaf(o[j][k], o[j][k], sum[0]);
                }
                if (ok[j]) store_pack<T, VEC>(a.out, base + c, o[j]);
            }
            if (!NEXT) continue;
            row_sum<1>(sum, red, a.TY, turn);
            r = rsqrtf(fmaf(sum[0], a.inv_cg, a.eps));
        }
        #pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (ty + j * a.TY) * VEC;
            float w[VEC];
            row_weights<VEC>(a.w2, ch0 + c, ok[j], w);
            #pragma unroll
            for (int k = 0; k < VEC; ++k) o[j][k] *= r * w[k];
            if (ok[j]) store_pack<T, VEC>(a.next, base + c, o[j]);
        }
    }
}

// Backward: block b walks images (b / G) Z + z, ... of group b % G; its channel sums go to
// part[b / G][channel], and gridDim / G images' worth on, the branch's.
template <typename T, int VEC, int NV, bool POST, bool NEXT>
__global__ void __launch_bounds__(kRowThreads, POST || NV * VEC > kRowHeld ? 1 : 2) block_bwd_row_kernel(const BlockArgs a)
{
    extern __shared__ __align__(16) float seats[];   // Z rows of a block's sums
    __shared__ float red[2 * 2 * (kRowThreads / 32)];
    const int ty = threadIdx.x % a.TY, z = threadIdx.x / a.TY;
    const int g = blockIdx.x % a.G, walker = blockIdx.x / a.G, walkers = gridDim.x / a.G, images = a.rows / a.G;
    const int ch0 = g * a.Cg, C = a.G * a.Cg;
    int turn = 0;
    float acc2[NV][VEC], acck[NV][VEC];
    #pragma unroll
    for (int j = 0; j < NV; ++j)
        #pragma unroll
        for (int k = 0; k < VEC; ++k) acc2[j][k] = acck[j][k] = 0.f;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    for (unsigned n0 = walker * a.Z; n0 < (unsigned)images; n0 += walkers * a.Z) {
        const unsigned n = n0 + z;
        const bool live = n < (unsigned)images;   // no row: r and m are 0, so that it adds nothing to the channel sums
        const int64_t base = (int64_t)n * C + ch0;
        Pack<T, VEC> pd[NV], px[NV], pg[NV], ph[NV], pz[NV];
        bool ok[NV];
        #pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (ty + j * a.TY) * VEC;
            ok[j] = live && c < a.Cg;
            pd[j] = row_load<T, VEC>(a.dout, base + c, ok[j]);
            if (NEXT) px[j] = row_load<T, VEC>(a.x, base + c, ok[j]);
            if (NEXT) pg[j] = row_load<T, VEC>(a.dnext, base + c, ok[j]);
            if (POST) ph[j] = row_load<T, VEC>(a.h, base + c, ok[j]);
            if (POST) pz[j] = row_load<T, VEC>(a.z, base + c, ok[j]);
        }
        float d[NV][VEC], sum[2] = {0.f, 0.f};
        float r = 0.f, m = 0.f;
        if (NEXT) {
            #pragma unroll
            for (int j = 0; j < NV; ++j) {
                float w[VEC];
                row_weights<VEC>(a.w2, ch0 + (ty + j * a.TY) * VEC, ok[j], w);
                #pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    const float x = to_f(px[j].v[k]);
                    d[j][k] = to_f(pg[j].v[k]) * w[k];
                    sum[0] = fmaf(x, x, sum[0]);
                    sum[1] = fmaf(x, d[j][k], sum[1]);
                }
            }
            row_sum<2>(sum, red, a.TY, turn);
            r = live ? rsqrtf(fmaf(sum[0], a.inv_cg, a.eps)) : 0.f;
            m = -sum[1] * a.inv_cg * r * r * r;   // from the left: r^3 alone may leave fp32
        }
        sum[0] = sum[1] = 0.f;
        #pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (ty + j * a.TY) * VEC;
            #pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float t = to_f(pd[j].v[k]);
                if (NEXT) {
                    const float x = to_f(px[j].v[k]);
                    d[j][k] = fmaf(x, m, fmaf(r, d[j][k], t));
                    acc2[j][k] = fmaf(to_f(pg[j].v[k]) * r, x, acc2[j][k]);
                } else {
                    d[j][k] = t;
                }
            }
            if (NEXT && ok[j]) store_pack<T, VEC>(a.dx, base + c, d[j]);
            if (POST) {
                float kc[VEC];
                branch_weights<VEC>(a, ch0 + c, ok[j], kc);
                #pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    const float h = to_f(ph[j].v[k]);
                    if (a.gate != GCONV_GATE_NONE) kc[k] *= gate_value(to_f(pz[j].v[k]), a.act);
                    sum[0] = fmaf(h, h, sum[0]);
                    sum[1] = fmaf(h, d[j][k] * kc[k], sum[1]);
                }
            }
        }
        if (!POST) continue;
        row_sum<2>(sum, red, a.TY, turn);
        r = live ? rsqrtf(fmaf(sum[0], a.inv_cg, a.eps)) : 0.f;
        m = -sum[1] * a.inv_cg * r * r * r;
        #pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (ty + j * a.TY) * VEC;
            float kc[VEC], dz[VEC];
            branch_weights<VEC>(a, ch0 + c, ok[j], kc);
            #pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float h = to_f(ph[j].v[k]), dr = d[j][k] * r, u = dr * h;
                float gv = 1.f, dg = 0.f;
                if (a.gate != GCONV_GATE_NONE) dg = gate_grad(to_f(pz[j].v[k]), a.act, &gv);
                acck[j][k] = fmaf(u, gv, acck[j][k]);
                dz[k] = u * kc[k] * dg;
                d[j][k] = fmaf(h, m, dr * kc[k] * gv);
            }
            if (!ok[j]) continue;
            store_pack<T, VEC>(a.dh, base + c, d[j]);
            if (!a.dz) continue;
            if (a.gate == GCONV_GATE_CHANNEL) row_floats<VEC>(static_cast<float *>(a.dz) + base + c, dz);
            else store_pack<T, VEC>(a.dz, base + c, dz);
        }
    }
    // the rows' sums in row order
    auto put = [&](const float (&acc)[NV][VEC], float *part) {
        if (a.Z > 1) {
            __syncthreads();
            #pragma unroll
            for (int j = 0; j < NV; ++j)
                #pragma unroll
                for (int k = 0; k < VEC; ++k) seats[((z * NV + j) * VEC + k) * a.TY + ty] = acc[j][k];
            __syncthreads();
            if (z > 0) return;
        }
        #pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (ty + j * a.TY) * VEC;
            if (c >= a.Cg) continue;
            float v[VEC];
            #pragma unroll
            for (int k = 0; k < VEC; ++k) {
                v[k] = acc[j][k];
                for (int i = 1; i < a.Z; ++i) v[k] += seats[((i * NV + j) * VEC + k) * a.TY + ty];
            }
            row_floats<VEC>(part + (int64_t)walker * C + ch0 + c, v);
        }
    };
    if (NEXT) put(acc2, a.part);
    if (POST) put(acck, a.part + (int64_t)walkers * C);
}

}  // namespace gconv
