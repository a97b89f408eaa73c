// block_norm.cuh -- what the block norm and block join kernels share, and those for very wide groups;
// the others are in block_stage.cuh.
//
// With r(t) = 1 / sqrt(mean over a group's channels of t^2 + eps), per image and position:
//   norm   y    = x r(x) w
//   join   out  = res + s act(z) (h r(h) w),      next = out r(out) w2
// and, for a gradient g of u = t r(t) w,
//   dt = r (g w) - t r^3 mean(g w t),             dw = sum over images and positions of g t r
// so one sweep gives the two sums mean(t^2) and mean(g w t), and nothing of the forward
// pass has to be kept but its inputs.
//
// Layout.  Image n's group g is a "row": a contiguous [Cg][P] matrix (P = H W) at element
// (n G + g) Cg P.  The sums run down its columns.  A block holds Z rows x TX vectors of VEC
// positions; a vector's channels are dealt over TY threads, NCH to a thread, so that a
// warp's loads are TX VEC consecutive positions of 32 / TX channels.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace gconv {

struct BlockArgs {
    int G, Cg, rows;          // rows = N G
    int P;                    // positions of a plane
    int TX, TY, Z;            // the block's shape; TX is a power of two
    int tiles, splits;        // tiles of TX vectors in a plane; blocks that share a row (backward)
    // staged kernels: a tile is PT positions of Z rows (flat: Z whole rows, tiles = 1)
    int PT, flat, per, total; // tiles a block walks, tiles in all
    int stages;               // tiles in shared memory: 2, or 1
    int cluster, Cc;          // blocks that share a group's channels, and how many each has
    int pitch, tensor;        // bytes of a staged channel, of a staged tensor
    // a tile of a tensor as boxes of its map, as 16-byte pieces of each channel, or (neither) as one run of
    // memory
    int boxes, box_rows, box_bytes;
    int pieces;
    int64_t bytes;            // of a whole tensor
    unsigned int *err;
    uint64_t wait_ns;
    int gate, act;
    float eps, inv_cg;
    const void *x, *h, *z;    // x: norm input / join residual (forward), join `out` (backward)
    const float *w, *s, *w2;  // branch weight, branch scale, weight of the (next) norm
    void *out, *next;         // forward results
    const void *dout, *dnext; // gradients of out (norm: residual branch) and of the norm's result
    void *dx, *dh, *dz;
    float *part;              // backward: [2][splits][N C] channel sums of next-norm and branch
};

// Threads that share the adding of one column sum: about the square root of its terms.
__host__ __device__ __forceinline__ int column_shares(int TY)
{
    int s = 1;
    while (s * s * 4 <= TY) s <<= 1;
    return s;
}

// The tensors of a staged launch as [N C][P] matrices, for tiles that are boxes of them.
struct StageMaps { CUtensorMap m[5]; };

__device__ __forceinline__ void from_f(float v, float *o) { *o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16 *o) { *o = __float2bfloat16_rn(v); }

template <typename T, int VEC>
__device__ __forceinline__ void store_pack(void *p, int64_t i, const float (&v)[VEC])
{
    Pack<T, VEC> o;
    #pragma unroll
    for (int k = 0; k < VEC; ++k) from_f(v[k], &o.v[k]);
    *reinterpret_cast<Pack<T, VEC> *>(static_cast<T *>(p) + i) = o;
}

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// act(z) and its derivative
__device__ __forceinline__ float gate_value(float z, int act)
{
    if (act == GCONV_ACT_NONE) return z;
    const float sg = sigmoid(z);
    return act == GCONV_ACT_SIGMOID ? sg : z * sg;
}

__device__ __forceinline__ float gate_grad(float z, int act, float *value)
{
    if (act == GCONV_ACT_NONE) { *value = z; return 1.f; }
    const float sg = sigmoid(z);
    if (act == GCONV_ACT_SIGMOID) { *value = sg; return sg * (1.f - sg); }
    *value = z * sg;
    return sg * (1.f + z * (1.f - sg));
}

// Adds v over the TY threads that share a row and a vector; every one of them gets the sum, by
// the same additions in the same order.  Through shared memory in two stages: TY / (NS VEC)
// threads a value add a share of the TY terms each, then every thread adds the shares.  (Shuffles
// cost one instruction a value and level, more than the stores and loads here.)
// `red`: Z (TY + shares) TX VEC NS floats.  The next call may follow at once: it writes what
// this one reads last only behind its own first barrier.
template <int NS, int VEC>
__device__ __forceinline__ void column_sum(float (&v)[NS][VEC], float *red, const BlockArgs &a, int tx, int ty, int z)
{
    if (a.TY == 1) return;
    const int width = a.TX * VEC * NS, shares = column_shares(a.TY);
    float *mine = red + z * (a.TY + shares) * width;
    #pragma unroll
    for (int q = 0; q < NS; ++q)
        *reinterpret_cast<Pack<float, VEC> *>(mine + ty * width + (q * a.TX + tx) * VEC) =
            *reinterpret_cast<Pack<float, VEC> *>(&v[q][0]);
    __syncthreads();
    float *sums = mine + a.TY * width;
    for (int i = ty * a.TX + tx; i < shares * width; i += a.TY * a.TX) {
        const int share = i / width, at = i - share * width;
        float t = 0.f;
        #pragma unroll 4
        for (int k = share; k < a.TY; k += shares) t += mine[k * width + at];
        sums[i] = t;
    }
    __syncthreads();
    #pragma unroll
    for (int q = 0; q < NS; ++q) {
        #pragma unroll
        for (int k = 0; k < VEC; ++k) v[q][k] = 0.f;
        for (int s = 0; s < shares; ++s) {
            const Pack<float, VEC> p = *reinterpret_cast<const Pack<float, VEC> *>(sums + s * width + (q * a.TX + tx) * VEC);
            #pragma unroll
            for (int k = 0; k < VEC; ++k) v[q][k] += p.v[k];
        }
    }
}

__device__ __forceinline__ float branch_coeff(const BlockArgs &a, int ch)
{
    return (a.w ? a.w[ch] : 1.f) * (a.s ? a.s[ch] : 1.f);
}

// ---- groups too wide for the staged kernels (a channel's 16 bytes times C / G beyond a cluster of
// eight blocks' shared memory): 32 positions a block, the channels walked in steps, inputs read again
// in each sweep, which the L2 serves in part.  Rare, and kept simple: norm of [8,32768,14,14] bf16
// 610 us (1220 with 32 positions a block on 56 of the SMs), 0.34 TB/s, bound by latency. ----

// out of the join at one element, from its three inputs; the roundings as in the staged kernel, so
// that out has the same bits with and without `next`
template <typename T>
__device__ __forceinline__ float walk_out(const BlockArgs &a, int64_t at, int ch, int64_t nc, float r)
{
    float g = branch_coeff(a, ch);
    if (a.gate == GCONV_GATE_FULL) g = __fmul_rn(g, gate_value(to_f(static_cast<const T *>(a.z)[at]), a.act));
    if (a.gate == GCONV_GATE_CHANNEL) g = __fmul_rn(g, gate_value(to_f(static_cast<const T *>(a.z)[nc]), a.act));
    return fmaf(g, __fmul_rn(to_f(static_cast<const T *>(a.h)[at]), r), to_f(static_cast<const T *>(a.x)[at]));
}

template <typename T>
__device__ __forceinline__ void walk_store(void *p, int64_t at, float v)
{
    const float q[1] = {v};
    store_pack<T, 1>(p, at, q);
}

template <typename T, bool POST, bool NEXT>
__global__ void __launch_bounds__(512) block_fwd_walk_kernel(const BlockArgs a)
{
    extern __shared__ __align__(16) float red[];
    const int tx = threadIdx.x % a.TX, ry = threadIdx.x / a.TX;
    const int ty = ry % a.TY, z = ry / a.TY;
    const int tile = blockIdx.x % a.tiles;
    const int row = (blockIdx.x / a.tiles) * a.Z + z;
    const int v0 = tile * a.TX + tx;
    const bool live = row < a.rows && v0 < a.P;
    const int64_t base = (int64_t)row * a.Cg * a.P + v0;
    const int ch0 = (row % a.G) * a.Cg;
    const int64_t nc0 = (int64_t)row * a.Cg;
    const int last = live ? a.Cg : 0;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    float sum[1][1] = {{0.f}};
    float r1 = 0.f;
    if (POST) {
        #pragma unroll 8
        for (int c = ty; c < last; c += a.TY) {
            const float t = to_f(static_cast<const T *>(a.h)[base + (int64_t)c * a.P]);
            sum[0][0] = fmaf(t, t, sum[0][0]);
        }
        column_sum<1, 1>(sum, red, a, tx, ty, z);
        r1 = rsqrtf(sum[0][0] * a.inv_cg + a.eps);
    }
    sum[0][0] = 0.f;
    #pragma unroll 4
    for (int c = ty; c < last; c += a.TY) {
        const int64_t at = base + (int64_t)c * a.P;
        const float t = POST ? walk_out<T>(a, at, ch0 + c, nc0 + c, r1) : to_f(static_cast<const T *>(a.x)[at]);
        sum[0][0] = fmaf(t, t, sum[0][0]);
        if (POST) walk_store<T>(a.out, at, t);
    }
    if (!NEXT) return;
    column_sum<1, 1>(sum, red, a, tx, ty, z);
    const float r2 = rsqrtf(sum[0][0] * a.inv_cg + a.eps);
    #pragma unroll 4
    for (int c = ty; c < last; c += a.TY) {
        const int64_t at = base + (int64_t)c * a.P;
        const float t = POST ? walk_out<T>(a, at, ch0 + c, nc0 + c, r1) : to_f(static_cast<const T *>(a.x)[at]);
        walk_store<T>(a.next, at, t * r2 * (a.w2 ? a.w2[ch0 + c] : 1.f));
    }
}

// The whole gradient of out at one element: dout, and what comes through the norm of x.
template <typename T, bool NEXT>
__device__ __forceinline__ float walk_grad(const BlockArgs &a, int64_t at, int ch, float r, float m, float *unit_grad)
{
    float d = a.dout ? to_f(static_cast<const T *>(a.dout)[at]) : 0.f;
    if (NEXT) {
        const float x = to_f(static_cast<const T *>(a.x)[at]), rg = to_f(static_cast<const T *>(a.dnext)[at]) * r;
        d = fmaf(-x, m, fmaf(rg, a.w2 ? a.w2[ch] : 1.f, d));
        *unit_grad = rg * x;
    }
    return d;
}

// One tile a block (splits = tiles); the channel sums of the tile go to `part`.
template <typename T, bool POST, bool NEXT>
__global__ void __launch_bounds__(512) block_bwd_walk_kernel(const BlockArgs a)
{
    extern __shared__ __align__(16) float red[];
    const int tx = threadIdx.x % a.TX, ry = threadIdx.x / a.TX;
    const int ty = ry % a.TY, z = ry / a.TY;
    const int split = blockIdx.x % a.splits;
    const int row = (blockIdx.x / a.splits) * a.Z + z;
    const int v0 = split * a.TX + tx;
    const bool row_ok = row < a.rows, live = row_ok && v0 < a.P;
    const int64_t base = (int64_t)row * a.Cg * a.P + v0;
    const int ch0 = (row % a.G) * a.Cg;
    const int64_t nc0 = (int64_t)row * a.Cg, NC = (int64_t)a.rows * a.Cg;
    const int last = live ? a.Cg : 0;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    float sum[2][1] = {{0.f}, {0.f}};
    float r2 = 0.f, m2 = 0.f;
    if (NEXT) {
        #pragma unroll 4
        for (int c = ty; c < last; c += a.TY) {
            const int64_t at = base + (int64_t)c * a.P;
            const float x = to_f(static_cast<const T *>(a.x)[at]);
            sum[0][0] = fmaf(x, x, sum[0][0]);
            sum[1][0] = fmaf(x, to_f(static_cast<const T *>(a.dnext)[at]) * (a.w2 ? a.w2[ch0 + c] : 1.f), sum[1][0]);
        }
        column_sum<2, 1>(sum, red, a, tx, ty, z);
        r2 = rsqrtf(sum[0][0] * a.inv_cg + a.eps);
        m2 = sum[1][0] * a.inv_cg * r2 * r2 * r2;
    }
    sum[0][0] = sum[1][0] = 0.f;
    // every thread goes round as often, with a channel or without: the sums over positions are shuffles
    // of whole warps, which hold several channels where TX is below 32
    for (int c0 = 0; c0 < a.Cg; c0 += a.TY) {
        const int c = c0 + ty;
        float unit_grad = 0.f;
        if (live && c < a.Cg) {
            const int64_t at = base + (int64_t)c * a.P;
            const float d = walk_grad<T, NEXT>(a, at, ch0 + c, r2, m2, &unit_grad);
            if (NEXT) walk_store<T>(a.dx, at, d);
            if (POST) {
                const float h = to_f(static_cast<const T *>(a.h)[at]);
                float g = branch_coeff(a, ch0 + c);
                if (a.gate == GCONV_GATE_FULL) g *= gate_value(to_f(static_cast<const T *>(a.z)[at]), a.act);
                if (a.gate == GCONV_GATE_CHANNEL) g *= gate_value(to_f(static_cast<const T *>(a.z)[nc0 + c]), a.act);
                sum[0][0] = fmaf(h, h, sum[0][0]);
                sum[1][0] = fmaf(h, d * g, sum[1][0]);
            }
        }
        if (NEXT) {
            for (int k = 1; k < a.TX; k <<= 1) unit_grad += __shfl_xor_sync(0xffffffffu, unit_grad, k);
            if (tx == 0 && row_ok && c < a.Cg) a.part[split * NC + nc0 + c] = unit_grad;
        }
    }
    if (!POST) return;
    column_sum<2, 1>(sum, red, a, tx, ty, z);
    const float r1 = rsqrtf(sum[0][0] * a.inv_cg + a.eps);
    const float m1 = sum[1][0] * a.inv_cg * r1 * r1 * r1;
    for (int c0 = 0; c0 < a.Cg; c0 += a.TY) {
        const int c = c0 + ty;
        float acc = 0.f;
        if (live && c < a.Cg) {
            const int64_t at = base + (int64_t)c * a.P;
            float unused;
            const float d = walk_grad<T, NEXT>(a, at, ch0 + c, r2, m2, &unused);
            const float h = to_f(static_cast<const T *>(a.h)[at]), kc = branch_coeff(a, ch0 + c);
            float g = 1.f, dg = 0.f;
            if (a.gate == GCONV_GATE_FULL) dg = gate_grad(to_f(static_cast<const T *>(a.z)[at]), a.act, &g);
            if (a.gate == GCONV_GATE_CHANNEL) g = gate_value(to_f(static_cast<const T *>(a.z)[nc0 + c]), a.act);
            const float dr = d * r1;
            acc = dr * h * (a.gate == GCONV_GATE_FULL ? g : 1.f);
            walk_store<T>(a.dh, at, fmaf(-h, m1, dr * kc * g));
            if (a.gate == GCONV_GATE_FULL && a.dz) walk_store<T>(a.dz, at, dr * kc * h * dg);
        }
        for (int k = 1; k < a.TX; k <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, k);
        if (tx == 0 && row_ok && c < a.Cg) a.part[(a.splits + split) * NC + nc0 + c] = acc;
    }
}

}  // namespace gconv
