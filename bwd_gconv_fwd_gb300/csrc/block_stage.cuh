// block_stage.cuh -- the block norm / join kernels for groups whose tiles fit in shared memory
// twice: while a block computes one tile, the next lands by 16-byte asynchronous copies.
//
// These operators do 4 to 40 operations an element against 4 to 16 bytes, so the memory is the
// limit as long as enough of it is in flight: a whole tile of every input here (40 to 100 KB an
// SM), where loads into registers end with each tile's reduction.  A copy moves aligned 16-byte
// pieces whatever the plane's size: a channel whose positions start off a 16-byte boundary is
// copied from the boundary before it, and read from where it starts in shared memory.
// What is left is the number of instructions, so two positions go through each arithmetic
// instruction (packed fp32 pairs) and every index is 32 bits and steps by constants.
//
// Two forms of a tile: PT positions of every channel of Z rows, or (flat) Z whole rows, which are
// one run of memory, for planes of at most 64 positions.  A lane holds two positions of nch
// channels: neighbours where P is even (one access for both), else TX apart.
#pragma once

#include "block_norm.cuh"

namespace gconv {

constexpr int kStageChannels = 8;

// ---- pairs of fp32 ------------------------------------------------------------------

struct F2 { uint64_t v; };

__device__ __forceinline__ F2 f2(float x, float y)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 parts(F2 a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// 1 / (1 + e^-z) of both: the error is that of the base-2 exponential's and the reciprocal's
// approximations, a few units in the last place.
__device__ __forceinline__ F2 sigmoid2(F2 z)
{
    const float2 t = parts(mul2(z, f2(-1.4426950408889634f)));
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    const float2 d = parts(add2(f2(e.x, e.y), f2(1.f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(d.y));
    return f2(e.x, e.y);
}

// ---- tiles --------------------------------------------------------------------------

// A tile: Z rows from row0, PT positions from p0.
struct Tile {
    int row0, p0;
    __device__ __forceinline__ void set(const BlockArgs &a, int t) { row0 = t / a.tiles * a.Z; p0 = t % a.tiles * a.PT; }
    __device__ __forceinline__ void next(const BlockArgs &a)
    {
        p0 += a.PT;
        if (p0 >= a.P) { p0 = 0; row0 += a.Z; }
    }
};

// Starts the copies of one tile of NT tensors to `dst` (a.tensor bytes each; a null tensor is skipped).
template <typename T, int NT>
__device__ __forceinline__ void stage_tile(const BlockArgs &a, const Tile &w, const char *const (&src)[NT], uint32_t dst)
{
    constexpr int es = (int)sizeof(T);
    const int rows = min(a.Z, a.rows - w.row0) * a.Cg;         // channels
    const int64_t first = (int64_t)w.row0 * a.Cg * a.P * es;
    auto copy = [&](uint32_t to, int64_t from) {
        const uint32_t n = (uint32_t)min((int64_t)16, a.bytes - from);
        #pragma unroll
        for (int i = 0; i < NT; ++i)
            if (src[i]) ptx::cp_async16(to + i * a.tensor, src[i] + from, n);
    };
    if (a.flat) {
        const int64_t lo = first & ~(int64_t)15;
        const int len = (int)(first - lo) + rows * a.P * es;
        for (int i = threadIdx.x * 16; i < len; i += blockDim.x * 16) copy(dst + i, lo + i);
    } else {
        const int k = threadIdx.x & (a.lanes2 - 1);
        int c = threadIdx.x / a.lanes2;
        const int step = blockDim.x / a.lanes2, len = min(a.PT, a.P - w.p0) * es;
        if (k >= a.pieces) return;
        int64_t at = first + ((int64_t)c * a.P + w.p0) * es;
        const int64_t hop = (int64_t)step * a.P * es;
        #pragma unroll 2
        for (; c < rows; c += step, at += hop) {
            const int off = 16 * k - (int)(at & 15);           // of the piece, from the channel's first position
            if (off < len) copy(dst + c * a.pitch + 16 * k, at + off);
        }
    }
}

// Two positions of a staged channel, as they lie next to each other (PAIR) or `apart` bytes apart.
template <typename T, bool PAIR>
__device__ __forceinline__ F2 read_two(const uint8_t *at, int apart)
{
    if constexpr (PAIR && sizeof(T) == 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(at);
        return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else if constexpr (PAIR) {
        F2 r;
        r.v = *reinterpret_cast<const uint64_t *>(at);
        return r;
    } else {
        return f2(to_f(*reinterpret_cast<const T *>(at)), to_f(*reinterpret_cast<const T *>(at + apart)));
    }
}

template <typename T, bool PAIR>
__device__ __forceinline__ void write_two(void *p, uint32_t i, int apart, F2 v, bool ok0, bool ok1)
{
    const float2 f = parts(v);
    if constexpr (PAIR) {
        const float o[2] = {f.x, f.y};
        if (ok0) store_pack<T, 2>(p, i, o);
    } else {
        T *q = static_cast<T *>(p) + i;
        if (ok0) from_f(f.x, q);
        if (ok1) from_f(f.y, q + apart);
    }
}

// column_sum for pairs; the widths are powers of two.
template <int NS>
__device__ __forceinline__ void column_sum2(F2 (&v)[NS], float *red, const BlockArgs &a, int tx, int ty, int z)
{
    if (a.TY == 1) return;
    const int pairs = a.TX * NS, lg = 31 - __clz(pairs);
    uint64_t *mine = reinterpret_cast<uint64_t *>(red) + z * (a.TY + a.shares) * pairs;
    #pragma unroll
    for (int q = 0; q < NS; ++q) mine[ty * pairs + q * a.TX + tx] = v[q].v;
    __syncthreads();
    uint64_t *sums = mine + a.TY * pairs;
    for (int i = ty * a.TX + tx; i < a.shares << lg; i += a.TY * a.TX) {
        const uint64_t *p = mine + (i & (pairs - 1));
        F2 t = f2(0.f);
        #pragma unroll 4
        for (int k = i >> lg; k < a.TY; k += a.shares) t = add2(t, F2{p[k << lg]});
        sums[i] = t.v;
    }
    __syncthreads();
    #pragma unroll
    for (int q = 0; q < NS; ++q) {
        F2 t{sums[q * a.TX + tx]};
        for (int s = 1; s < a.shares; ++s) t = add2(t, F2{sums[(s << lg) + q * a.TX + tx]});
        v[q] = t;
    }
}

// r = 1 / sqrt(mean + eps) of both positions; 0 at a dead one, where eps = 0 would make it infinite.
__device__ __forceinline__ F2 root2(const BlockArgs &a, F2 sum, bool ok0, bool ok1)
{
    const float2 s = parts(sum);
    const float x = rsqrtf(fmaf(s.x, a.inv_cg, a.eps)), y = rsqrtf(fmaf(s.y, a.inv_cg, a.eps));
    return f2(ok0 ? x : 0.f, ok1 ? y : 0.f);
}

// A thread's place: vector tx, channels ty, ty + TY, ... of row z of the tile, and from it the
// offsets of its first channel and the steps to the next.  (32 bits: the low four bits of a
// byte address survive, and a tensor has fewer than 2^31 elements.)
struct Seat {
    int tx, ty, z, pos, c0;
    int apart, s_first, s_step, m_step;
    uint32_t e_step;
};

template <typename T, bool PAIR>
__device__ __forceinline__ Seat seat(const BlockArgs &a)
{
    constexpr int es = (int)sizeof(T);
    Seat s;
    s.tx = threadIdx.x % a.TX;
    const int ry = threadIdx.x / a.TX;
    s.ty = ry % a.TY;
    s.z = ry / a.TY;
    s.pos = PAIR ? 2 * s.tx : s.tx;
    s.c0 = s.z * a.Cg + s.ty;
    s.apart = PAIR ? 1 : a.TX;
    s.s_first = s.c0 * a.pitch + s.pos * es;
    s.s_step = a.TY * a.pitch;
    s.m_step = a.flat ? 0 : a.TY * a.P * es;
    s.e_step = (uint32_t)(a.TY * a.P);
    return s;
}

template <typename T>
__device__ __forceinline__ int staged_at(const Seat &s, uint32_t m0, int j)
{
    return s.s_first + j * s.s_step + (int)((m0 + (uint32_t)(j * s.m_step)) & 15u);
}

// Byte offset, modulo 16, of the thread's first channel in this tile (flat: of the tile).
template <typename T>
__device__ __forceinline__ uint32_t misfit(const BlockArgs &a, const Seat &s, const Tile &w)
{
    const uint32_t first = (uint32_t)w.row0 * (uint32_t)a.Cg * (uint32_t)a.P;
    return (first + (a.flat ? 0u : (uint32_t)s.c0 * (uint32_t)a.P + (uint32_t)w.p0)) * (uint32_t)sizeof(T);
}

template <typename T, bool PAIR, bool POST, bool NEXT>
__global__ void __launch_bounds__(512) block_fwd_stage_kernel(const BlockArgs a)
{
    constexpr int NT = POST ? 3 : 1, NCH = kStageChannels;
    extern __shared__ __align__(128) uint8_t smem[];
    float *red = reinterpret_cast<float *>(smem + 2 * NT * a.tensor);
    const Seat s = seat<T, PAIR>(a);
    const int apart = s.apart * (int)sizeof(T);
    const bool full = POST && a.gate == GCONV_GATE_FULL;
    const char *src[NT];
    src[0] = static_cast<const char *>(a.x);
    if constexpr (POST) { src[1] = static_cast<const char *>(a.h); src[2] = full ? static_cast<const char *>(a.z) : nullptr; }
    const uint32_t stage0 = ptx::smem_u32(smem);
    const int t0 = blockIdx.x * a.per, t1 = min(a.total, t0 + a.per);
    Tile w, ahead;
    w.set(a, t0);
    ahead = w;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    stage_tile<T, NT>(a, ahead, src, stage0);
    ptx::cp_async_commit();

    int at_row = -1;
    float kb[NCH], wn[NCH];
    for (int t = t0; t < t1; ++t, w.next(a)) {
        const int buf = (t - t0) & 1;
        ptx::cp_async_wait_group<0>();
        __syncthreads();
        if (t + 1 < t1) {
            ahead.next(a);
            stage_tile<T, NT>(a, ahead, src, stage0 + (buf ^ 1) * NT * a.tensor);
            ptx::cp_async_commit();
        }
        const uint8_t *st = smem + buf * NT * a.tensor;
        const bool in_row = w.row0 + s.z < a.rows;
        const bool ok0 = in_row && w.p0 + s.pos < a.P, ok1 = in_row && w.p0 + s.pos + s.apart < a.P;
        if (at_row != w.row0) {
            at_row = w.row0;
            const int row = w.row0 + s.z, ch0 = (row % a.G) * a.Cg + s.ty;
            #pragma unroll
            for (int j = 0; j < NCH; ++j) {
                kb[j] = wn[j] = 0.f;
                if (in_row && s.ty + j * a.TY < a.Cg) {
                    if (NEXT) wn[j] = a.w2 ? a.w2[ch0 + j * a.TY] : 1.f;
                    if (POST) {
                        kb[j] = branch_coeff(a, ch0 + j * a.TY);
                        if (a.gate == GCONV_GATE_CHANNEL)
                            kb[j] = __fmul_rn(kb[j], gate_value(to_f(static_cast<const T *>(a.z)[(int64_t)row * a.Cg + s.ty + j * a.TY]), a.act));
                    }
                }
            }
        }
        const uint32_t m0 = misfit<T>(a, s, w);
        const uint32_t e0 = ((uint32_t)w.row0 * (uint32_t)a.Cg + (uint32_t)s.c0) * (uint32_t)a.P + (uint32_t)(w.p0 + s.pos);
        int at[NCH];
        F2 sum[1] = {f2(0.f)};
        F2 o[NCH];
        #pragma unroll
        for (int j = 0; j < NCH; ++j) {
            at[j] = staged_at<T>(s, m0, j);
            if (s.ty + j * a.TY < a.Cg) {
                o[j] = read_two<T, PAIR>(st + (POST ? a.tensor : 0) + at[j], apart);
                sum[0] = fma2(o[j], o[j], sum[0]);
            }
        }
        column_sum2<1>(sum, red, a, s.tx, s.ty, s.z);
        F2 r = root2(a, sum[0], true, true);
        if (POST) {
            sum[0] = f2(0.f);
            #pragma unroll
            for (int j = 0; j < NCH; ++j)
                if (s.ty + j * a.TY < a.Cg) {
                    const F2 x = read_two<T, PAIR>(st + at[j], apart);
                    F2 g = f2(kb[j]);
                    if (full) {
                        const F2 z = read_two<T, PAIR>(st + 2 * a.tensor + at[j], apart);
                        const F2 sg = sigmoid2(z);
                        const F2 v = a.act == GCONV_ACT_NONE ? z : a.act == GCONV_ACT_SIGMOID ? sg : mul2(z, sg);
                        g = mul2(g, v);
                    }
                    o[j] = fma2(g, mul2(o[j], r), x);
                    write_two<T, PAIR>(a.out, e0 + j * s.e_step, s.apart, o[j], ok0, ok1);
                    sum[0] = fma2(o[j], o[j], sum[0]);
                }
            if (!NEXT) continue;
            column_sum2<1>(sum, red, a, s.tx, s.ty, s.z);
            r = root2(a, sum[0], true, true);
        }
        #pragma unroll
        for (int j = 0; j < NCH; ++j)
            if (s.ty + j * a.TY < a.Cg)
                write_two<T, PAIR>(a.next, e0 + j * s.e_step, s.apart, mul2(o[j], mul2(r, f2(wn[j]))), ok0, ok1);
    }
}

// Backward.  A block walks consecutive tiles; its channel sums of a block of rows stay in
// registers and go to part[i][row][channel] when the rows change, i counting the blocks that
// share those rows.  Dead positions hold what an earlier tile left: they meet no live one but in
// the channel sums, which leave them out.
template <typename T, bool PAIR, bool POST, bool NEXT>
__global__ void __launch_bounds__(512) block_bwd_stage_kernel(const BlockArgs a)
{
    constexpr int NT = POST && NEXT ? 5 : 3, NCH = kStageChannels;
    extern __shared__ __align__(128) uint8_t smem[];
    float *red = reinterpret_cast<float *>(smem + 2 * NT * a.tensor);
    const Seat s = seat<T, PAIR>(a);
    const int apart = s.apart * (int)sizeof(T);
    const bool full = POST && a.gate == GCONV_GATE_FULL;
    const char *src[NT];
    src[0] = static_cast<const char *>(a.dout);
    constexpr int iX = 1, iG = 2, iH = NEXT ? 3 : 1, iZ = NEXT ? 4 : 2;
    if constexpr (NEXT) { src[iX] = static_cast<const char *>(a.x); src[iG] = static_cast<const char *>(a.dnext); }
    if constexpr (POST) { src[iH] = static_cast<const char *>(a.h); src[iZ] = full ? static_cast<const char *>(a.z) : nullptr; }
    const uint32_t stage0 = ptx::smem_u32(smem);
    const int t0 = blockIdx.x * a.per, t1 = min(a.total, t0 + a.per);
    const int64_t NC = (int64_t)a.rows * a.Cg;
    Tile w, ahead;
    w.set(a, t0);
    ahead = w;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    stage_tile<T, NT>(a, ahead, src, stage0);
    ptx::cp_async_commit();

    int at_row = -1;
    bool in_row = false;
    float acc2[NCH], acck[NCH], wn[NCH], kb[NCH];
    auto flush = [&] {
        const int share = blockIdx.x - (int)((int64_t)(at_row / a.Z) * a.tiles / a.per);
        float *p0 = a.part + share * NC + (int64_t)(at_row + s.z) * a.Cg + s.ty;
        #pragma unroll
        for (int j = 0; j < NCH; ++j)
            if (j < a.nch) {
                float s2 = acc2[j], sk = acck[j];
                for (int m = 1; m < a.TX; m <<= 1) {
                    if (NEXT) s2 += __shfl_xor_sync(0xffffffffu, s2, m);
                    if (POST) sk += __shfl_xor_sync(0xffffffffu, sk, m);
                }
                if (s.tx == 0 && in_row && s.ty + j * a.TY < a.Cg) {
                    if (NEXT) p0[j * a.TY] = s2;
                    if (POST) p0[a.splits * NC + j * a.TY] = sk;
                }
            }
    };
    for (int t = t0; t < t1; ++t, w.next(a)) {
        const int buf = (t - t0) & 1;
        ptx::cp_async_wait_group<0>();
        __syncthreads();
        if (t + 1 < t1) {
            ahead.next(a);
            stage_tile<T, NT>(a, ahead, src, stage0 + (buf ^ 1) * NT * a.tensor);
            ptx::cp_async_commit();
        }
        const uint8_t *st = smem + buf * NT * a.tensor;
        if (at_row != w.row0) {
            if (at_row >= 0) flush();
            at_row = w.row0;
            in_row = w.row0 + s.z < a.rows;
            const int row = w.row0 + s.z, ch0 = (row % a.G) * a.Cg + s.ty;
            #pragma unroll
            for (int j = 0; j < NCH; ++j) {
                acc2[j] = acck[j] = wn[j] = kb[j] = 0.f;
                if (in_row && s.ty + j * a.TY < a.Cg) {
                    if (NEXT) wn[j] = a.w2 ? a.w2[ch0 + j * a.TY] : 1.f;
                    if (POST) kb[j] = branch_coeff(a, ch0 + j * a.TY);
                    if (POST && a.gate == GCONV_GATE_CHANNEL)
                        kb[j] *= gate_value(to_f(static_cast<const T *>(a.z)[(int64_t)row * a.Cg + s.ty + j * a.TY]), a.act);
                }
            }
        }
        const bool ok0 = in_row && w.p0 + s.pos < a.P, ok1 = in_row && w.p0 + s.pos + s.apart < a.P;
        const uint32_t m0 = misfit<T>(a, s, w);
        const uint32_t e0 = ((uint32_t)w.row0 * (uint32_t)a.Cg + (uint32_t)s.c0) * (uint32_t)a.P + (uint32_t)(w.p0 + s.pos);
        int at[NCH];
        #pragma unroll
        for (int j = 0; j < NCH; ++j) at[j] = staged_at<T>(s, m0, j);
        F2 d[NCH], sum[2] = {f2(0.f), f2(0.f)};
        F2 r = f2(0.f), m = f2(0.f);   // r, and -mean(g w t) r^3
        if (NEXT) {
            #pragma unroll
            for (int j = 0; j < NCH; ++j)
                if (s.ty + j * a.TY < a.Cg) {
                    const F2 x = read_two<T, PAIR>(st + iX * a.tensor + at[j], apart);
                    const F2 g = read_two<T, PAIR>(st + iG * a.tensor + at[j], apart);
                    sum[0] = fma2(x, x, sum[0]);
                    sum[1] = fma2(x, mul2(g, f2(wn[j])), sum[1]);
                }
            column_sum2<2>(sum, red, a, s.tx, s.ty, s.z);
            r = root2(a, sum[0], ok0, ok1);
            m = mul2(mul2(sum[1], f2(-a.inv_cg)), mul2(r, mul2(r, r)));
        }
        sum[0] = sum[1] = f2(0.f);
        F2 sg[NCH];   // the gate's sigmoid, or its value without one
        #pragma unroll
        for (int j = 0; j < NCH; ++j)
            if (s.ty + j * a.TY < a.Cg) {
                d[j] = f2(0.f);
                if (a.dout) d[j] = read_two<T, PAIR>(st + at[j], apart);
                if (NEXT) {
                    const F2 x = read_two<T, PAIR>(st + iX * a.tensor + at[j], apart);
                    const F2 g = mul2(read_two<T, PAIR>(st + iG * a.tensor + at[j], apart), r);
                    d[j] = fma2(x, m, fma2(g, f2(wn[j]), d[j]));
                    const float2 u = parts(mul2(g, x));
                    if (ok0) acc2[j] += u.x;
                    if (ok1) acc2[j] += u.y;
                    write_two<T, PAIR>(a.dx, e0 + j * s.e_step, s.apart, d[j], ok0, ok1);
                }
                if (POST) {
                    const F2 h = read_two<T, PAIR>(st + iH * a.tensor + at[j], apart);
                    F2 v = mul2(d[j], f2(kb[j]));
                    if (full) {
                        const F2 z = read_two<T, PAIR>(st + iZ * a.tensor + at[j], apart);
                        sg[j] = sigmoid2(z);
                        if (a.act == GCONV_ACT_NONE) sg[j] = z;
                        v = mul2(v, a.act == GCONV_ACT_SILU ? mul2(z, sg[j]) : sg[j]);
                    }
                    sum[0] = fma2(h, h, sum[0]);
                    sum[1] = fma2(h, v, sum[1]);
                }
            }
        if (!POST) continue;
        column_sum2<2>(sum, red, a, s.tx, s.ty, s.z);
        r = root2(a, sum[0], ok0, ok1);
        m = mul2(mul2(sum[1], f2(-a.inv_cg)), mul2(r, mul2(r, r)));
        #pragma unroll
        for (int j = 0; j < NCH; ++j)
            if (s.ty + j * a.TY < a.Cg) {
                const uint32_t e = e0 + j * s.e_step;
                const F2 h = read_two<T, PAIR>(st + iH * a.tensor + at[j], apart);
                const F2 dr = mul2(d[j], r), dk = mul2(dr, f2(kb[j]));
                F2 u = mul2(dr, h), dh = dk;   // the channel gate is in kb; its own gradient needs u without it
                if (full) {
                    // act'(z): 1; s (1 - s); s (1 + z (1 - s)) = s + g (1 - s)
                    F2 g = sg[j], dg = f2(1.f);
                    if (a.act != GCONV_ACT_NONE) {
                        const F2 rest = fma2(sg[j], f2(-1.f), f2(1.f));
                        if (a.act == GCONV_ACT_SILU) {
                            g = mul2(read_two<T, PAIR>(st + iZ * a.tensor + at[j], apart), sg[j]);
                            dg = fma2(g, rest, sg[j]);
                        } else {
                            dg = mul2(g, rest);
                        }
                    }
                    if (a.dz) write_two<T, PAIR>(a.dz, e, s.apart, mul2(mul2(dk, h), dg), ok0, ok1);
                    u = mul2(u, g);
                    dh = mul2(dk, g);
                }
                const float2 q = parts(u);
                if (ok0) acck[j] += q.x;
                if (ok1) acck[j] += q.y;
                write_two<T, PAIR>(a.dh, e, s.apart, fma2(h, m, dh), ok0, ok1);
            }
    }
    if (at_row >= 0) flush();
}

}  // namespace gconv
