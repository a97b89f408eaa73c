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
    int gate, act;
    float eps, inv_cg;
    const void *x, *h, *z;    // x: norm input / join residual (forward), join `out` (backward)
    const float *w, *s, *w2;  // branch weight, branch scale, weight of the (next) norm
    void *out, *next;         // forward results
    const void *dout, *dnext; // gradients of out (norm: residual branch) and of the norm's result
    void *dx, *dh, *dz;
    float *part;              // backward: [2][splits][N C] channel sums of next-norm and branch
};

// VEC elements of T as they lie in memory.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack { T v[VEC]; };

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

// act(z) and its derivative
__device__ __forceinline__ float gate_value(float z, int act)
{
    if (act == GCONV_ACT_NONE) return z;
    const float sg = __fdividef(1.f, 1.f + __expf(-z));
    return act == GCONV_ACT_SIGMOID ? sg : z * sg;
}

__device__ __forceinline__ float gate_grad(float z, int act, float *value)
{
    if (act == GCONV_ACT_NONE) { *value = z; return 1.f; }
    const float sg = __fdividef(1.f, 1.f + __expf(-z));
    if (act == GCONV_ACT_SIGMOID) { *value = sg; return sg * (1.f - sg); }
    *value = z * sg;
    return sg * (1.f + z * (1.f - sg));
}

// Adds v over the TY threads that share a row and a vector; every one of them gets the sum.
// Lanes of a warp that differ in ty are added by shuffles, the warps of a row through
// shared memory, always in the same order.  `red`: Z * ceil(TX TY / 32) * TX * VEC * NS floats.
template <int NS, int VEC>
__device__ __forceinline__ void column_sum(float (&v)[NS][VEC], float *red, const BlockArgs &a, int tx, int ty, int z)
{
    const int per_row = a.TX * a.TY;
    const int top = per_row < 32 ? per_row : 32;
    for (int m = a.TX; m < top; m <<= 1) {
        #pragma unroll
        for (int q = 0; q < NS; ++q)
            #pragma unroll
            for (int k = 0; k < VEC; ++k) v[q][k] += __shfl_xor_sync(0xffffffffu, v[q][k], m);
    }
    if (per_row <= 32) return;
    const int warps = per_row >> 5, width = a.TX * VEC * NS;
    float *mine = red + (int64_t)z * (warps + 1) * width;
    const int in_row = ty * a.TX + tx;
    if ((in_row & 31) < a.TX) {
        #pragma unroll
        for (int q = 0; q < NS; ++q)
            #pragma unroll
            for (int k = 0; k < VEC; ++k) mine[(in_row >> 5) * width + (q * VEC + k) * a.TX + tx] = v[q][k];
    }
    __syncthreads();
    for (int i = in_row; i < width; i += per_row) {
        float t = 0.f;
        for (int w = 0; w < warps; ++w) t += mine[w * width + i];
        mine[warps * width + i] = t;
    }
    __syncthreads();
    #pragma unroll
    for (int q = 0; q < NS; ++q)
        #pragma unroll
        for (int k = 0; k < VEC; ++k) v[q][k] = mine[warps * width + (q * VEC + k) * a.TX + tx];
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

// Forward.  POST: the join's branch; NEXT: the norm (of out, or of x alone without POST).
// ONE: a thread's NCH channels are all of its share; else it walks its share in steps of
// TY NCH channels and reads the inputs again in each sweep.
template <typename T, int VEC, int NCH, bool POST, bool NEXT, bool ONE>
__global__ void __launch_bounds__(512) block_fwd_kernel(const BlockArgs a)
{
    extern __shared__ float red[];
    const int tx = threadIdx.x % a.TX, ry = threadIdx.x / a.TX;
    const int ty = ry % a.TY, z = ry / a.TY;
    const int tile = blockIdx.x % a.tiles;
    const int row = (blockIdx.x / a.tiles) * a.Z + z;
    const int v0 = tile * a.TX + tx;
    const bool live = row < a.rows && v0 < a.PV;
    const int64_t base = (int64_t)row * a.Cg * a.P + (int64_t)v0 * VEC;
    const int ch0 = live ? (row % a.G) * a.Cg : 0;             // first channel of the row's group
    const int64_t nc0 = live ? (int64_t)row * a.Cg : 0;        // first element of the row in [N][C]
    const int step = a.TY * NCH;
    const int span = ONE ? 1 : (a.Cg + step - 1) / step;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    float sum[1][VEC];
    float r1[VEC];
    Pack<T, VEC> hk[NCH], xk[NCH];
    if (POST) {
        #pragma unroll
        for (int k = 0; k < VEC; ++k) sum[0][k] = 0.f;
        for (int cc = 0; cc < span; ++cc) {
            #pragma unroll
            for (int j = 0; j < NCH; ++j) {
                const int c = cc * step + j * a.TY + ty;
                if (live && c < a.Cg) {
                    hk[j] = load_pack<T, VEC>(a.h, base + (int64_t)c * a.P);
                    if (ONE) xk[j] = load_pack<T, VEC>(a.x, base + (int64_t)c * a.P);
                }
            }
            #pragma unroll
            for (int j = 0; j < NCH; ++j) {
                const int c = cc * step + j * a.TY + ty;
                if (live && c < a.Cg) {
                    #pragma unroll
                    for (int k = 0; k < VEC; ++k) { const float t = to_f(hk[j].v[k]); sum[0][k] = fmaf(t, t, sum[0][k]); }
                }
            }
        }
        column_sum<1, VEC>(sum, red, a, tx, ty, z);
        #pragma unroll
        for (int k = 0; k < VEC; ++k) r1[k] = rsqrtf(sum[0][k] * a.inv_cg + a.eps);
        __syncthreads();
    }
    // out, and the sum of its squares
    float o[NCH][VEC];
    #pragma unroll
    for (int k = 0; k < VEC; ++k) sum[0][k] = 0.f;
    for (int cc = 0; cc < span; ++cc) {
        #pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = cc * step + j * a.TY + ty;
            if (!live || c >= a.Cg) continue;
            const int64_t at = base + (int64_t)c * a.P;
            if (!POST || !ONE) xk[j] = load_pack<T, VEC>(a.x, at);
            if (POST && !ONE) hk[j] = load_pack<T, VEC>(a.h, at);
            Pack<T, VEC> zk;
            float zc = 0.f;
            if (POST && a.gate == GCONV_GATE_FULL) zk = load_pack<T, VEC>(a.z, at);
            if (POST && a.gate == GCONV_GATE_CHANNEL) zc = gate_value(to_f(static_cast<const T *>(a.z)[nc0 + c]), a.act);
            const float kc = POST ? branch_coeff(a, ch0 + c) : 0.f;
            #pragma unroll
            for (int k = 0; k < VEC; ++k) {
                float t = to_f(xk[j].v[k]);
                if (POST) {
                    const float g = a.gate == GCONV_GATE_FULL ? gate_value(to_f(zk.v[k]), a.act)
                                  : a.gate == GCONV_GATE_CHANNEL ? zc : 1.f;
                    t = join_sum(t, kc, g, to_f(hk[j].v[k]), r1[k]);
                }
                o[j][k] = t;
                sum[0][k] = fmaf(t, t, sum[0][k]);
            }
            if (POST) store_pack<T, VEC>(a.out, at, o[j]);
        }
    }
    if (!NEXT) return;
    column_sum<1, VEC>(sum, red, a, tx, ty, z);
    float r2[VEC];
    #pragma unroll
    for (int k = 0; k < VEC; ++k) r2[k] = rsqrtf(sum[0][k] * a.inv_cg + a.eps);
    for (int cc = 0; cc < span; ++cc) {
        #pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = cc * step + j * a.TY + ty;
            if (!live || c >= a.Cg) continue;
            const int64_t at = base + (int64_t)c * a.P;
            if (!ONE) {
                const Pack<T, VEC> xr = load_pack<T, VEC>(a.x, at);
                Pack<T, VEC> hr, zr;
                float zc = 0.f;
                if (POST) hr = load_pack<T, VEC>(a.h, at);
                if (POST && a.gate == GCONV_GATE_FULL) zr = load_pack<T, VEC>(a.z, at);
                if (POST && a.gate == GCONV_GATE_CHANNEL) zc = gate_value(to_f(static_cast<const T *>(a.z)[nc0 + c]), a.act);
                const float kc = POST ? branch_coeff(a, ch0 + c) : 0.f;
                #pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    o[j][k] = to_f(xr.v[k]);
                    if (POST) {
                        const float g = a.gate == GCONV_GATE_FULL ? gate_value(to_f(zr.v[k]), a.act)
                                      : a.gate == GCONV_GATE_CHANNEL ? zc : 1.f;
                        o[j][k] = join_sum(o[j][k], kc, g, to_f(hr.v[k]), r1[k]);
                    }
                }
            }
            const float wc = a.w2 ? a.w2[ch0 + c] : 1.f;
            float y[VEC];
            #pragma unroll
            for (int k = 0; k < VEC; ++k) y[k] = o[j][k] * r2[k] * wc;
            store_pack<T, VEC>(a.next, at, y);
        }
    }
}

// Backward.  NEXT: dx = dout + gradient of the norm of x (= out); POST: the branch's dh, dz
// from dx (= dout without NEXT).  Channel sums of a block's share go to `part`.  With ONE a
// block walks the tiles split, split + splits, ... of its rows and keeps its channel sums in
// registers; else there is one split a tile.
template <typename T, int VEC, int NCH, bool POST, bool NEXT, bool ONE>
__global__ void __launch_bounds__(512) block_bwd_kernel(const BlockArgs a)
{
    extern __shared__ float red[];
    const int tx = threadIdx.x % a.TX, ry = threadIdx.x / a.TX;
    const int ty = ry % a.TY, z = ry / a.TY;
    const int split = blockIdx.x % a.splits;
    const int row = (blockIdx.x / a.splits) * a.Z + z;
    const bool row_ok = row < a.rows;
    const int ch0 = row_ok ? (row % a.G) * a.Cg : 0;
    const int64_t nc0 = row_ok ? (int64_t)row * a.Cg : 0;
    const int step = a.TY * NCH;
    const int span = ONE ? 1 : (a.Cg + step - 1) / step;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    float acc2[NCH], acck[NCH];
    #pragma unroll
    for (int j = 0; j < NCH; ++j) acc2[j] = acck[j] = 0.f;

    // the gradient that reaches `out` at one element of channel c
    for (int tile = split; tile < a.tiles; tile += a.splits) {
        const int v0 = tile * a.TX + tx;
        const bool live = row_ok && v0 < a.PV;
        const int64_t base = (int64_t)row * a.Cg * a.P + (int64_t)v0 * VEC;
        Pack<T, VEC> xk[NCH], gk[NCH];
        float r2[VEC], m2[VEC];
        if (NEXT) {
            float sum[2][VEC];
            #pragma unroll
            for (int k = 0; k < VEC; ++k) sum[0][k] = sum[1][k] = 0.f;
            for (int cc = 0; cc < span; ++cc) {
                #pragma unroll
                for (int j = 0; j < NCH; ++j) {
                    const int c = cc * step + j * a.TY + ty;
                    if (!live || c >= a.Cg) continue;
                    xk[j] = load_pack<T, VEC>(a.x, base + (int64_t)c * a.P);
                    gk[j] = load_pack<T, VEC>(a.dnext, base + (int64_t)c * a.P);
                }
                #pragma unroll
                for (int j = 0; j < NCH; ++j) {
                    const int c = cc * step + j * a.TY + ty;
                    if (!live || c >= a.Cg) continue;
                    const float wc = a.w2 ? a.w2[ch0 + c] : 1.f;
                    #pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        const float t = to_f(xk[j].v[k]);
                        sum[0][k] += t * t;
                        sum[1][k] += t * (to_f(gk[j].v[k]) * wc);
                    }
                }
            }
            column_sum<2, VEC>(sum, red, a, tx, ty, z);
            #pragma unroll
            for (int k = 0; k < VEC; ++k) {
                r2[k] = rsqrtf(sum[0][k] * a.inv_cg + a.eps);
                m2[k] = sum[1][k] * a.inv_cg * r2[k] * r2[k] * r2[k];
            }
            __syncthreads();
        }
        // dx, and the branch's two sums
        float d[NCH][VEC];
        Pack<T, VEC> hk[NCH], zk[NCH];
        float sum[2][VEC];
        #pragma unroll
        for (int k = 0; k < VEC; ++k) sum[0][k] = sum[1][k] = 0.f;
        for (int cc = 0; cc < span; ++cc) {
            #pragma unroll
            for (int j = 0; j < NCH; ++j) {
                const int c = cc * step + j * a.TY + ty;
                float acc = 0.f;
                if (live && c < a.Cg) {
                    const int64_t at = base + (int64_t)c * a.P;
                    Pack<T, VEC> dk;
                    if (a.dout) dk = load_pack<T, VEC>(a.dout, at);
                    if (NEXT && !ONE) {
                        xk[j] = load_pack<T, VEC>(a.x, at);
                        gk[j] = load_pack<T, VEC>(a.dnext, at);
                    }
                    if (POST) {
                        hk[j] = load_pack<T, VEC>(a.h, at);
                        if (a.gate == GCONV_GATE_FULL) zk[j] = load_pack<T, VEC>(a.z, at);
                    }
                    const float wc = NEXT && a.w2 ? a.w2[ch0 + c] : 1.f;
                    #pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        float t = a.dout ? to_f(dk.v[k]) : 0.f;
                        if (NEXT) {
                            const float xv = to_f(xk[j].v[k]), gv = to_f(gk[j].v[k]);
                            t += r2[k] * (gv * wc) - xv * m2[k];
                            acc += gv * (xv * r2[k]);
                        }
                        d[j][k] = t;
                    }
                    if (NEXT) store_pack<T, VEC>(a.dx, at, d[j]);
                    if (POST) {
                        const float kc = branch_coeff(a, ch0 + c);
                        const float zc = a.gate == GCONV_GATE_CHANNEL
                                       ? gate_value(to_f(static_cast<const T *>(a.z)[nc0 + c]), a.act) : 1.f;
                        #pragma unroll
                        for (int k = 0; k < VEC; ++k) {
                            const float hv = to_f(hk[j].v[k]);
                            const float g = a.gate == GCONV_GATE_FULL ? gate_value(to_f(zk[j].v[k]), a.act) : zc;
                            sum[0][k] += hv * hv;
                            sum[1][k] += hv * (d[j][k] * kc * g);
                        }
                    }
                }
                if (ONE) acc2[j] += acc;
                else if (NEXT) {
                    for (int m = 1; m < a.TX; m <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
                    if (tx == 0 && row_ok && c < a.Cg) a.part[(int64_t)split * a.rows * a.Cg + nc0 + c] = acc;
                }
            }
        }
        if (!POST) { if (ONE) __syncthreads(); continue; }
        column_sum<2, VEC>(sum, red, a, tx, ty, z);
        float r1[VEC], m1[VEC];
        #pragma unroll
        for (int k = 0; k < VEC; ++k) {
            r1[k] = rsqrtf(sum[0][k] * a.inv_cg + a.eps);
            m1[k] = sum[1][k] * a.inv_cg * r1[k] * r1[k] * r1[k];
        }
        __syncthreads();
        for (int cc = 0; cc < span; ++cc) {
            #pragma unroll
            for (int j = 0; j < NCH; ++j) {
                const int c = cc * step + j * a.TY + ty;
                float acc = 0.f;
                if (live && c < a.Cg) {
                    const int64_t at = base + (int64_t)c * a.P;
                    if (!ONE) {
                        Pack<T, VEC> dk;
                        if (a.dout) dk = load_pack<T, VEC>(a.dout, at);
                        if (NEXT) {
                            xk[j] = load_pack<T, VEC>(a.x, at);
                            gk[j] = load_pack<T, VEC>(a.dnext, at);
                        }
                        hk[j] = load_pack<T, VEC>(a.h, at);
                        if (a.gate == GCONV_GATE_FULL) zk[j] = load_pack<T, VEC>(a.z, at);
                        const float wc = NEXT && a.w2 ? a.w2[ch0 + c] : 1.f;
                        #pragma unroll
                        for (int k = 0; k < VEC; ++k) {
                            d[j][k] = a.dout ? to_f(dk.v[k]) : 0.f;
                            if (NEXT) d[j][k] += r2[k] * (to_f(gk[j].v[k]) * wc) - to_f(xk[j].v[k]) * m2[k];
                        }
                    }
                    const float kc = branch_coeff(a, ch0 + c);
                    const float zc = a.gate == GCONV_GATE_CHANNEL
                                   ? gate_value(to_f(static_cast<const T *>(a.z)[nc0 + c]), a.act) : 1.f;
                    float dh[VEC], dz[VEC];
                    #pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        const float hv = to_f(hk[j].v[k]);
                        float g = zc, dg = 0.f;
                        if (a.gate == GCONV_GATE_FULL) dg = gate_grad(to_f(zk[j].v[k]), a.act, &g);
                        const float unit = hv * r1[k];
                        dh[k] = r1[k] * (d[j][k] * kc * g) - hv * m1[k];
                        dz[k] = d[j][k] * kc * unit * dg;
                        // the channel gate's own gradient needs the sum without the gate; the
                        // finish kernel multiplies it in
                        acc += d[j][k] * unit * (a.gate == GCONV_GATE_FULL ? g : 1.f);
                    }
                    store_pack<T, VEC>(a.dh, at, dh);
                    if (a.gate == GCONV_GATE_FULL && a.dz) store_pack<T, VEC>(a.dz, at, dz);
                }
                if (ONE) acck[j] += acc;
                else {
                    for (int m = 1; m < a.TX; m <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
                    if (tx == 0 && row_ok && c < a.Cg) a.part[(int64_t)(a.splits + split) * a.rows * a.Cg + nc0 + c] = acc;
                }
            }
        }
        if (ONE) __syncthreads();
    }
    if (!ONE) return;
    #pragma unroll
    for (int j = 0; j < NCH; ++j) {
        const int c = j * a.TY + ty;
        float s2 = acc2[j], sk = acck[j];
        for (int m = 1; m < a.TX; m <<= 1) {
            if (NEXT) s2 += __shfl_xor_sync(0xffffffffu, s2, m);
            if (POST) sk += __shfl_xor_sync(0xffffffffu, sk, m);
        }
        if (tx == 0 && row_ok && c < a.Cg) {
            if (NEXT) a.part[(int64_t)split * a.rows * a.Cg + nc0 + c] = s2;
            if (POST) a.part[(int64_t)(a.splits + split) * a.rows * a.Cg + nc0 + c] = sk;
        }
    }
}

}  // namespace gconv
