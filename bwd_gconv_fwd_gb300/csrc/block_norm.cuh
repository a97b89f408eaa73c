// block_norm.cuh -- device code of the block norm and block join kernels (block_norm.cu).
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
    int P, PV;                // positions of a plane, vectors of VEC positions in it
    int TX, TY, Z;            // the block's shape; TX is a power of two
    int tiles, splits;        // tiles of TX vectors in a plane; blocks that share a row (backward)
    // staged kernels: a tile is PT positions of Z rows (flat: Z whole rows, tiles = 1)
    int PT, flat, per, total; // tiles a block walks, tiles in all
    int pitch, tensor;        // bytes of a staged channel, of a staged tensor
    int pieces, lanes2;       // 16-byte pieces of a channel, and the power of two threads for them
    int64_t bytes;            // of a whole tensor
    int whole;                // bytes is a multiple of 16
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

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const void *p, int64_t i)
{
    return *reinterpret_cast<const Pack<T, VEC> *>(static_cast<const T *>(p) + i);
}

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

// res + k g (h r), each rounding written out: out has the same bits with and without `next`.
__device__ __forceinline__ float join_sum(float res, float k, float g, float h, float r)
{
    return fmaf(__fmul_rn(k, g), __fmul_rn(h, r), res);
}

// ---- a group's channels in the registers of one thread block ----------------------

// Forward.  POST: the join's branch; NEXT: the norm (of out, or of x alone without POST).
// Every load of a tile is issued before its first use and its first store: the stores may
// alias the loads as far as the compiler knows, and a load behind one would wait for it.
template <typename T, int VEC, int NCH, bool POST, bool NEXT>
__global__ void __launch_bounds__(512) block_fwd_kernel(const BlockArgs a)
{
    extern __shared__ __align__(16) float red[];
    const int tx = threadIdx.x % a.TX, ry = threadIdx.x / a.TX;
    const int ty = ry % a.TY, z = ry / a.TY;
    const int tile = blockIdx.x % a.tiles;
    const int row = (blockIdx.x / a.tiles) * a.Z + z;
    const int v0 = tile * a.TX + tx;
    const bool live = row < a.rows && v0 < a.PV;
    const int64_t base = (int64_t)row * a.Cg * a.P + (int64_t)v0 * VEC + (int64_t)ty * a.P;
    const int64_t hop = (int64_t)a.TY * a.P;                   // to the thread's next channel
    const int ch0 = live ? (row % a.G) * a.Cg + ty : 0;
    const int64_t nc0 = live ? (int64_t)row * a.Cg + ty : 0;   // in [N][C]
    const int mine = live ? (a.Cg - ty + a.TY - 1) / a.TY : 0; // channels of this thread, at most NCH
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    Pack<T, VEC> hk[NCH], xk[NCH], zk[NCH];
    float kb[NCH], wn[NCH];
    #pragma unroll
    for (int j = 0; j < NCH; ++j) {
        hk[j] = xk[j] = zk[j] = Pack<T, VEC>{};
        if (j < mine) {
            xk[j] = load_pack<T, VEC>(a.x, base + j * hop);
            if (POST) hk[j] = load_pack<T, VEC>(a.h, base + j * hop);
            if (POST && a.gate == GCONV_GATE_FULL) zk[j] = load_pack<T, VEC>(a.z, base + j * hop);
        }
    }
    #pragma unroll
    for (int j = 0; j < NCH; ++j) {
        kb[j] = wn[j] = 0.f;
        if (j < mine) {
            if (NEXT) wn[j] = a.w2 ? a.w2[ch0 + j * a.TY] : 1.f;
            if (POST) {
                kb[j] = branch_coeff(a, ch0 + j * a.TY);
                if (a.gate == GCONV_GATE_CHANNEL)
                    kb[j] = __fmul_rn(kb[j], gate_value(to_f(static_cast<const T *>(a.z)[nc0 + j * a.TY]), a.act));
            }
        }
    }
    float sum[1][VEC];
    float o[NCH][VEC];
    if (POST) {
        #pragma unroll
        for (int k = 0; k < VEC; ++k) sum[0][k] = 0.f;
        #pragma unroll
        for (int j = 0; j < NCH; ++j)
            #pragma unroll
            for (int k = 0; k < VEC; ++k) { const float t = to_f(hk[j].v[k]); sum[0][k] = fmaf(t, t, sum[0][k]); }
        column_sum<1, VEC>(sum, red, a, tx, ty, z);
        #pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const float r = rsqrtf(sum[0][k] * a.inv_cg + a.eps);
            #pragma unroll
            for (int j = 0; j < NCH; ++j) {
                const float g = a.gate == GCONV_GATE_FULL ? __fmul_rn(kb[j], gate_value(to_f(zk[j].v[k]), a.act)) : kb[j];
                o[j][k] = fmaf(g, __fmul_rn(to_f(hk[j].v[k]), r), to_f(xk[j].v[k]));
            }
        }
        #pragma unroll
        for (int j = 0; j < NCH; ++j)
            if (j < mine) store_pack<T, VEC>(a.out, base + j * hop, o[j]);
        if (!NEXT) return;
    } else {
        #pragma unroll
        for (int j = 0; j < NCH; ++j)
            #pragma unroll
            for (int k = 0; k < VEC; ++k) o[j][k] = to_f(xk[j].v[k]);
    }
    #pragma unroll
    for (int k = 0; k < VEC; ++k) sum[0][k] = 0.f;
    #pragma unroll
    for (int j = 0; j < NCH; ++j)
        #pragma unroll
        for (int k = 0; k < VEC; ++k) sum[0][k] = fmaf(o[j][k], o[j][k], sum[0][k]);
    column_sum<1, VEC>(sum, red, a, tx, ty, z);
    #pragma unroll
    for (int k = 0; k < VEC; ++k) {
        const float r = rsqrtf(sum[0][k] * a.inv_cg + a.eps);
        #pragma unroll
        for (int j = 0; j < NCH; ++j) o[j][k] *= r * wn[j];
    }
    #pragma unroll
    for (int j = 0; j < NCH; ++j)
        if (j < mine) store_pack<T, VEC>(a.next, base + j * hop, o[j]);
}

// Backward.  NEXT: dx = dout + gradient of the norm of x (= out); POST: the branch's dh, dz
// from dx (= dout without NEXT).  A block walks the tiles split, split + splits, ... of its
// rows and keeps its channel sums in registers; they go to `part` at the end.
template <typename T, int VEC, int NCH, bool POST, bool NEXT>
__global__ void __launch_bounds__(512) block_bwd_kernel(const BlockArgs a)
{
    extern __shared__ __align__(16) float red[];
    const int tx = threadIdx.x % a.TX, ry = threadIdx.x / a.TX;
    const int ty = ry % a.TY, z = ry / a.TY;
    const int split = blockIdx.x % a.splits;
    const int row = (blockIdx.x / a.splits) * a.Z + z;
    const bool row_ok = row < a.rows;
    const int64_t base0 = (int64_t)row * a.Cg * a.P + (int64_t)ty * a.P;
    const int64_t hop = (int64_t)a.TY * a.P;
    const int ch0 = row_ok ? (row % a.G) * a.Cg + ty : 0;
    const int64_t nc0 = row_ok ? (int64_t)row * a.Cg + ty : 0;
    const int mine_row = row_ok ? (a.Cg - ty + a.TY - 1) / a.TY : 0;
    const bool full = POST && a.gate == GCONV_GATE_FULL;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    float acc2[NCH], acck[NCH], wn[NCH], kb[NCH], zc[NCH];
    #pragma unroll
    for (int j = 0; j < NCH; ++j) {
        acc2[j] = acck[j] = wn[j] = kb[j] = 0.f;
        zc[j] = 1.f;
        if (j < mine_row) {
            if (NEXT) wn[j] = a.w2 ? a.w2[ch0 + j * a.TY] : 1.f;
            if (POST) kb[j] = branch_coeff(a, ch0 + j * a.TY);
            if (POST && a.gate == GCONV_GATE_CHANNEL)
                zc[j] = gate_value(to_f(static_cast<const T *>(a.z)[nc0 + j * a.TY]), a.act);
        }
    }
    for (int tile = split; tile < a.tiles; tile += a.splits) {
        const int v0 = tile * a.TX + tx;
        const int mine = v0 < a.PV ? mine_row : 0;
        const int64_t base = base0 + (int64_t)v0 * VEC;
        Pack<T, VEC> xk[NCH], gk[NCH], dk[NCH], hk[NCH], zk[NCH];
        #pragma unroll
        for (int j = 0; j < NCH; ++j) {
            xk[j] = gk[j] = dk[j] = hk[j] = zk[j] = Pack<T, VEC>{};
            if (j < mine) {
                const int64_t at = base + j * hop;
                if (NEXT) {
                    xk[j] = load_pack<T, VEC>(a.x, at);
                    gk[j] = load_pack<T, VEC>(a.dnext, at);
                }
                if (a.dout) dk[j] = load_pack<T, VEC>(a.dout, at);
                if (POST) hk[j] = load_pack<T, VEC>(a.h, at);
                if (full) zk[j] = load_pack<T, VEC>(a.z, at);
            }
        }
        float sum[2][VEC];
        float d[NCH][VEC];
        #pragma unroll
        for (int j = 0; j < NCH; ++j)
            #pragma unroll
            for (int k = 0; k < VEC; ++k) d[j][k] = to_f(dk[j].v[k]);
        if (NEXT) {
            #pragma unroll
            for (int k = 0; k < VEC; ++k) sum[0][k] = sum[1][k] = 0.f;
            #pragma unroll
            for (int j = 0; j < NCH; ++j)
                #pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    const float t = to_f(xk[j].v[k]);
                    sum[0][k] = fmaf(t, t, sum[0][k]);
                    sum[1][k] = fmaf(t, to_f(gk[j].v[k]) * wn[j], sum[1][k]);
                }
            column_sum<2, VEC>(sum, red, a, tx, ty, z);
            #pragma unroll
            for (int k = 0; k < VEC; ++k) {
                // r is 0 past the plane's end, where eps = 0 would make it infinite
                const float r = v0 < a.PV ? rsqrtf(sum[0][k] * a.inv_cg + a.eps) : 0.f;
                const float m = sum[1][k] * a.inv_cg * r * r * r;
                #pragma unroll
                for (int j = 0; j < NCH; ++j) {
                    const float x = to_f(xk[j].v[k]), rg = to_f(gk[j].v[k]) * r;
                    d[j][k] = fmaf(-x, m, fmaf(rg, wn[j], d[j][k]));
                    acc2[j] = fmaf(rg, x, acc2[j]);
                }
            }
            #pragma unroll
            for (int j = 0; j < NCH; ++j)
                if (j < mine) store_pack<T, VEC>(a.dx, base + j * hop, d[j]);
        }
        if (POST) {
            #pragma unroll
            for (int k = 0; k < VEC; ++k) sum[0][k] = sum[1][k] = 0.f;
            float sg[NCH][VEC];   // the gate's sigmoid, or its value without one
            #pragma unroll
            for (int j = 0; j < NCH; ++j)
                #pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    const float h = to_f(hk[j].v[k]), zv = to_f(zk[j].v[k]);
                    sg[j][k] = !full ? zc[j] : a.act == GCONV_ACT_NONE ? zv : sigmoid(zv);
                    const float g = full && a.act == GCONV_ACT_SILU ? zv * sg[j][k] : sg[j][k];
                    sum[0][k] = fmaf(h, h, sum[0][k]);
                    sum[1][k] = fmaf(h, d[j][k] * (kb[j] * g), sum[1][k]);
                }
            column_sum<2, VEC>(sum, red, a, tx, ty, z);
            #pragma unroll
            for (int k = 0; k < VEC; ++k) {
                // r is 0 past the plane's end, where eps = 0 would make it infinite
                const float r = v0 < a.PV ? rsqrtf(sum[0][k] * a.inv_cg + a.eps) : 0.f;
                const float m = sum[1][k] * a.inv_cg * r * r * r;
                #pragma unroll
                for (int j = 0; j < NCH; ++j) {
                    const float h = to_f(hk[j].v[k]), zv = to_f(zk[j].v[k]), s = sg[j][k];
                    const float g = full && a.act == GCONV_ACT_SILU ? zv * s : s;
                    const float dr = d[j][k] * r, dk_ = dr * kb[j];
                    // act'(z): 1; s (1 - s); s (1 + z (1 - s)) = s + g (1 - s)
                    const float dg = a.act == GCONV_ACT_NONE ? 1.f : a.act == GCONV_ACT_SIGMOID ? s - s * s : fmaf(g, 1.f - s, s);
                    // the channel gate's own gradient needs the sum without the gate; the
                    // finish kernel multiplies it in
                    acck[j] = fmaf(dr * h, full ? g : 1.f, acck[j]);
                    d[j][k] = fmaf(-h, m, dk_ * g);          // dh
                    sg[j][k] = dk_ * h * dg;                 // dz
                }
            }
            #pragma unroll
            for (int j = 0; j < NCH; ++j)
                if (j < mine) {
                    store_pack<T, VEC>(a.dh, base + j * hop, d[j]);
                    if (full && a.dz) store_pack<T, VEC>(a.dz, base + j * hop, sg[j]);
                }
        }
    }
    #pragma unroll
    for (int j = 0; j < NCH; ++j) {
        float s2 = acc2[j], sk = acck[j];
        for (int m = 1; m < a.TX; m <<= 1) {
            if (NEXT) s2 += __shfl_xor_sync(0xffffffffu, s2, m);
            if (POST) sk += __shfl_xor_sync(0xffffffffu, sk, m);
        }
        if (tx == 0 && j < mine_row) {
            if (NEXT) a.part[(int64_t)split * a.rows * a.Cg + nc0 + j * a.TY] = s2;
            if (POST) a.part[(int64_t)(a.splits + split) * a.rows * a.Cg + nc0 + j * a.TY] = sk;
        }
    }
}

// ---- groups too wide for that: the channels walked in steps, inputs read again in each sweep ----

// out of the join at one element, from its three inputs
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
    // every lane of a warp goes round as often: the sums over positions are shuffles
    for (int c = ty; c < a.Cg; c += a.TY) {
        float unit_grad = 0.f;
        if (live) {
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
            if (tx == 0 && row_ok) a.part[split * NC + nc0 + c] = unit_grad;
        }
    }
    if (!POST) return;
    column_sum<2, 1>(sum, red, a, tx, ty, z);
    const float r1 = rsqrtf(sum[0][0] * a.inv_cg + a.eps);
    const float m1 = sum[1][0] * a.inv_cg * r1 * r1 * r1;
    for (int c = ty; c < a.Cg; c += a.TY) {
        float acc = 0.f;
        if (live) {
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
        if (tx == 0 && row_ok) a.part[(a.splits + split) * NC + nc0 + c] = acc;
    }
}

}  // namespace gconv
