// scan.cuh -- what the selective scan's kernels share.
//
//   h[t] = exp(d[t] A) h[t-1] + d[t] u[t] B[t],   y[t] = sum_s C[t] h[t] + D u[t]
//
// for every sequence, channel and state s.  A thread holds K consecutive positions of a pair of channels in
// registers and walks over the states: the recurrence over its run starts from zero, a scan over the TL lanes
// that hold neighbouring runs of the same channels gives what enters each run, and a second walk makes the
// states.  The exponentials, one a state and position, are taken once.  What crosses from one tile of TL K
// positions to the next, and what enters a tile, stays in shared memory, as do B and C (in fp32, shared by all the
// channels of a block).  Both channels of a pair go through one instruction (packed fp32), the recurrences too; B and C
// are the same for both, which such an instruction takes from a single register.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace gconv {

constexpr int kScanMark = 64;       // positions between the states that the forward pass keeps for the gradient
constexpr int kScanStates = 16;     // states whose B and C are in shared memory at once
constexpr int kScanMaxStates = 256;
// Lanes along the positions and positions a lane: a tile is 64 positions of 8 channels a warp.  Longer runs take fewer
// scans but twice the registers (16 positions: [8,2048,2048] forward 384 us against 359), more lanes more steps a
// scan (32: 533 us), and fewer blocks each; where blocks are few, sequences are cut in pieces instead.
constexpr int kScanLanes = 8, kScanRun = 8, kScanTile = kScanLanes * kScanRun;
constexpr int kScanOwn = 32 / kScanLanes * 2;      // channels a warp

// Whether the forward pass keeps the sums before the gate for the gradient.  In fp32 it does; in bf16 the room that `saved` has for
// them would round a sum to 16 bits, and the gradient makes them again from its states.
template <typename T> constexpr bool scan_keeps = sizeof(T) == sizeof(float);

struct ScanArgs {
    int N, C, L, G, S, Cg;
    int softplus;
    int ncb, sets;              // blocks of channels in a group; channel sets that a block takes in turn (gradient)
    int chunks, chunk_tiles;    // pieces of a sequence that are scanned side by side, and the tiles of one
    int marks;                  // ceil(L / kScanMark)
    const void *u, *delta, *z, *B, *Cm;
    int64_t su, sdelta, sz, sB, sC, sy;
    const float *A, *D, *bias;
    const float *state;
    float *state_out;
    const int *lengths;
    void *y;
    float *mark;                // [N][marks][S][C]
    float *pre;                 // [N][C][L], y before the gate (fp32 activations)
    float *init;                // [N][chunks][S][C]: what enters a piece (chunks > 1)
    float *dsum;                // [N][chunks][C]: sum of d over a piece
    // gradient
    const void *dy;
    int64_t sdy, sdu, sddelta, sdz, sdB, sdC;
    void *du, *ddelta, *dz, *dB, *dC;
    const float *dstate_out;
    float *dstate;
    float *part;                // [N][G][ncb][2][S][L]: dB and dC of a block's channels (ncb > 1)
    float *pA, *pD, *pb;        // [N chunks][C][S], [N chunks][C], [N chunks][C]
};

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float scan_sigmoid(float x) { return rcp(1.f + ex2(x * -kLog2e)); }

// ---- pairs of channels ---------------------------------------------------------------

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 ex2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }
__device__ __forceinline__ float2 rcp(float2 x) { return make_float2(rcp(x.x), rcp(x.y)); }
__device__ __forceinline__ float2 operator*(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 operator+(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

__device__ __forceinline__ float2 scan_sigmoid(float2 x) { return rcp(both(1.f) + ex2(x * both(-kLog2e))); }

// log(1 + e^x) = max(x, 0) + log1p(e), e = e^-|x|.  The product with log2 e is carried in two parts, as its rounding
// alone would be |x| 2^-24 of a small result; log1p(e) = 2 atanh(e / (2 + e)) by its series, whose terms fall by
// nine at least (seven of them: 2^-25).
__device__ __forceinline__ float2 scan_softplus(float2 x)
{
    const float2 m = make_float2(fmaxf(-fabsf(x.x), -104.f), fmaxf(-fabsf(x.y), -104.f));
    const float2 hi = m * both(kLog2e);
    const float2 lo = fma2(m, both(kLog2e), make_float2(-hi.x, -hi.y));
    const float2 e0 = ex2(hi);
    const float2 e = fma2(e0, lo * both(kLn2), e0);
    const float2 s = e * rcp(both(2.f) + e), q = s * s;
    float2 r = fma2(q, both(1.f / 13.f), both(1.f / 11.f));
    r = fma2(q, r, both(1.f / 9.f));
    r = fma2(q, r, both(1.f / 7.f));
    r = fma2(q, r, both(1.f / 5.f));
    r = fma2(q, r, both(1.f / 3.f));
    r = fma2(q, r, both(1.f));
    r = fma2(s + s, r, make_float2(x.x > 0.f ? x.x : 0.f, x.y > 0.f ? x.y : 0.f));
    return make_float2(x.x == x.x ? r.x : x.x, x.y == x.y ? r.y : x.y);
}
__device__ __forceinline__ float scan_softplus(float x) { return scan_softplus(both(x)).x; }

// Where a thread's run lies within a sequence: positions t .. t + K - 1 of a pair of channels whose rows lie L apart,
// in 16-byte pieces where VEC (rows and t are multiples of that).  Pieces behind the row, and a second channel that is
// none, stand for others that are there, so that no load needs a condition; clear_run takes out what is not to be used.
template <typename T, int K, bool VEC>
struct Place {
    static constexpr int E = VEC ? 16 / (int)sizeof(T) : 1;
    int64_t x[VEC ? K / E : 1];     // of the first channel; the second's are `step` further
    int64_t step;
    int t, L;

    __device__ __forceinline__ Place(int64_t row, int t_, int L_, bool there0, bool there1) : step(there1 ? L_ : 0), t(t_), L(L_)
    {
        if (!there0) row = 0;
        if constexpr (VEC) {
            #pragma unroll
            for (int i = 0; i < K / E; ++i) x[i] = row + (t + i * E < L ? t + i * E : 0);
        } else {
            x[0] = row;
        }
    }
};

// A run's values as they lie in memory.  Loading and converting are apart so that all of a tile's loads are on their
// way before the first is waited for.
template <typename T, int K, bool VEC>
struct Run {
    static constexpr int E = VEC ? 16 / (int)sizeof(T) : 1;
    Pack<T, E> x[K / E], y[K / E];

    __device__ __forceinline__ void load(const T *base, const Place<T, K, VEC> &at)
    {
        if constexpr (VEC) {
            #pragma unroll
            for (int i = 0; i < K / E; ++i) {
                x[i] = *reinterpret_cast<const Pack<T, E> *>(base + at.x[i]);
                y[i] = *reinterpret_cast<const Pack<T, E> *>(base + at.x[i] + at.step);
            }
        } else {
            const T *p = base + at.x[0];
            const bool whole = at.t + K <= at.L;    // no element needs a place of its own
            if (whole) {
                p += at.t;
                #pragma unroll
                for (int i = 0; i < K; ++i) {
                    x[i].v[0] = p[i];
                    y[i].v[0] = p[at.step + i];
                }
            } else {
                #pragma unroll
                for (int i = 0; i < K; ++i) {
                    const int o = min(at.t + i, at.L - 1);
                    x[i].v[0] = p[o];
                    y[i].v[0] = p[at.step + o];
                }
            }
        }
    }
    __device__ __forceinline__ float2 at(int k) const { return make_float2(to_f(x[k / E].v[k % E]), to_f(y[k / E].v[k % E])); }
};

// Zeros from the ends on, whatever came before.
template <int K>
__device__ __forceinline__ void clear_run(int t, int end0, int end1, float2 (&v)[K])
{
    if (t + K <= min(end0, end1)) return;
    #pragma unroll
    for (int i = 0; i < K; ++i) {
        v[i].x = t + i < end0 ? v[i].x : 0.f;
        v[i].y = t + i < end1 ? v[i].y : 0.f;
    }
}

template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ void put2(float *to, float x, float y) { to[0] = x; to[1] = y; }
__device__ __forceinline__ void put2(__nv_bfloat16 *to, float x, float y)
{
    *reinterpret_cast<__nv_bfloat162 *>(to) = __floats2bfloat162_rn(x, y);
}

// The same, stored up to L positions of the channels that are there.
template <typename T, int K, bool VEC>
__device__ __forceinline__ void store_run(T *row, int64_t L, int t, bool there0, bool there1, const float2 (&v)[K])
{
    if constexpr (VEC) {
        constexpr int E = 16 / (int)sizeof(T);
        #pragma unroll
        for (int i = 0; i < K; i += E) {
            if (t + i >= L) continue;
            Pack<T, E> x, y;
            #pragma unroll
            for (int j = 0; j < E; j += 2) {
                put2(x.v + j, v[i + j].x, v[i + j + 1].x);
                put2(y.v + j, v[i + j].y, v[i + j + 1].y);
            }
            if (there0) *reinterpret_cast<Pack<T, E> *>(row + t + i) = x;
            if (there1) *reinterpret_cast<Pack<T, E> *>(row + L + t + i) = y;
        }
    } else {
        if (t + K <= L) {
            if (there0) {
                #pragma unroll
                for (int i = 0; i < K; ++i) row[t + i] = from_f<T>(v[i].x);
            }
            if (there1) {
                #pragma unroll
                for (int i = 0; i < K; ++i) row[L + t + i] = from_f<T>(v[i].y);
            }
        } else {
            #pragma unroll
            for (int i = 0; i < K; ++i) {
                if (t + i >= L) continue;
                if (there0) row[t + i] = from_f<T>(v[i].x);
                if (there1) row[L + t + i] = from_f<T>(v[i].y);
            }
        }
    }
}

// Place of position t of a tile in a row of shared memory: four floats of gap after every 32, so that eight lanes
// eight positions apart read 16 bytes each without meeting in a bank.  A run of 8 has no gap inside.
__device__ __forceinline__ int spot(int t) { return t + ((t >> 5) << 2); }
constexpr int spots(int TT) { return TT + (TT / 32) * 4; }

// B or C of up to kScanStates states, in fp32, zeros from `end` on: loaded first, stored to shared memory later.  The positions
// are those of the lanes' runs, kScanLanes of kScanRun each, the first at t0 and each `each` further (kScanRun: 64 neighbours).
template <typename T, bool VEC>
struct States {
    static constexpr int E = VEC ? 16 / (int)sizeof(T) : 1, PER = kScanTile / E;
    static constexpr int ALL = kScanStates * PER / 128, HELD = ALL < 1 ? 1 : ALL < 8 ? ALL : 8;   // pieces a thread holds; more are stored as they come
    Pack<T, E> x[HELD];

    __device__ __forceinline__ static int place(int i, int t0, int each)
    {
        const int t = (i % PER) * E;
        return t0 + t / kScanRun * each + t % kScanRun;
    }
    __device__ __forceinline__ static void put(float *sh, int i, int t0, int each, int end, const Pack<T, E> &v)
    {
        const int left = end - place(i, t0, each);
        float *to = sh + (i / PER) * spots(kScanTile) + spot((i % PER) * E);
        if constexpr (VEC) {
            float f[E];
            #pragma unroll
            for (int j = 0; j < E; ++j) f[j] = to_f(v.v[j]);
            if (left < E) {
                #pragma unroll
                for (int j = 0; j < E; ++j) f[j] = j < left ? f[j] : 0.f;
            }
            #pragma unroll
            for (int j = 0; j < E; j += 4) *reinterpret_cast<float4 *>(to + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
        } else {
            *to = to_f(v.v[0]);
        }
    }
    __device__ __forceinline__ static Pack<T, E> get(const T *base, int64_t L, int i, int t0, int each, int end)
    {
        Pack<T, E> v{};
        const int t = place(i, t0, each);
        if (t < end) v = *reinterpret_cast<const Pack<T, E> *>(base + (i / PER) * L + t);
        return v;
    }
    __device__ __forceinline__ void load(const T *base, int64_t L, int count, int t0, int each, int end)
    {
        #pragma unroll
        for (int j = 0; j < HELD; ++j) {
            const int i = threadIdx.x + j * blockDim.x;
            x[j] = i < count * PER ? get(base, L, i, t0, each, end) : Pack<T, E>{};
        }
    }
    __device__ __forceinline__ void store(const T *base, int64_t L, int count, int t0, int each, int end, float *sh) const
    {
        #pragma unroll
        for (int j = 0; j < HELD; ++j) {
            const int i = threadIdx.x + j * blockDim.x;
            if (i < count * PER) put(sh, i, t0, each, end, x[j]);
        }
        for (int i = threadIdx.x + HELD * blockDim.x; i < count * PER; i += blockDim.x)
            put(sh, i, t0, each, end, get(base, L, i, t0, each, end));
    }
};

// Asks for the line at a pointer, ahead of its load.
__device__ __forceinline__ void fetch(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <int K>
__device__ __forceinline__ void read_run(const float *row, float (&v)[K])
{
    #pragma unroll
    for (int i = 0; i < K; i += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(row + i);
        v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
    }
}

__device__ __forceinline__ float2 shift_up(float2 v, int o, int width)
{
    return make_float2(__shfl_up_sync(~0u, v.x, o, width), __shfl_up_sync(~0u, v.y, o, width));
}
__device__ __forceinline__ float2 shift_down(float2 v, int o, int width)
{
    return make_float2(__shfl_down_sync(~0u, v.x, o, width), __shfl_down_sync(~0u, v.y, o, width));
}
__device__ __forceinline__ float2 pick(bool c, float2 a, float2 b) { return make_float2(c ? a.x : b.x, c ? a.y : b.y); }

// A log2 e, finite, so that a step of zero leaves a state as it was even where A is not (where A is NaN, a sequence without
// positions takes 0 in its place).
__device__ __forceinline__ float decay_rate(float a)
{
    const float v = a * kLog2e;
    return v != v ? v : fminf(fmaxf(v, -3.4e38f), 3.4e38f);
}

__device__ __forceinline__ int sequence_end(const ScanArgs &a, int n)
{
    if (!a.lengths) return a.L;
    const int v = a.lengths[n];
    return v < 0 ? 0 : v < a.L ? v : a.L;
}

}  // namespace gconv
