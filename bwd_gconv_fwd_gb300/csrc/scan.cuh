// scan.cuh -- what the selective scan's kernels share.
//
//   h[t] = exp(d[t] A) h[t-1] + d[t] u[t] B[t],   y[t] = sum_s C[t] h[t] + D u[t]
//
// for every sequence, channel and state s.  A thread holds K consecutive positions of P channels in
// registers and walks over the states: the recurrence over its run starts from zero, a scan over the TL lanes
// that hold neighbouring runs of the same channels gives what enters each run, and a second walk makes the
// states.  The exponentials, one a state and position, are taken once.  What crosses from one tile of TL K
// positions to the next, and what enters a tile, stays in shared memory, as do B and C (in fp32, shared by all the
// channels of a block).
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace gconv {

constexpr int kScanMark = 64;       // positions between the states that the forward pass keeps for the gradient
constexpr int kScanStates = 16;     // states whose B and C are in shared memory at once
constexpr int kScanMaxStates = 256;

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
    void *pre;                  // [N][C][L], y before the gate
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

// log(1 + e^x) = max(x, 0) + log1p(e), e = e^-|x|.  The product with log2 e is carried in two parts, as its rounding
// alone would be |x| 2^-24 of a small result; log1p(e) = 2 atanh(e / (2 + e)) by its series, whose terms fall by
// nine at least (seven of them: 2^-25).
__device__ __forceinline__ float scan_softplus(float x)
{
    const float m = fmaxf(-fabsf(x), -104.f);
    const float hi = m * kLog2e;
    const float lo = fmaf(m, kLog2e, -hi);
    const float e0 = ex2(hi);
    const float e = fmaf(e0, lo * kLn2, e0);
    const float s = e * rcp(2.f + e), q = s * s;
    float r = fmaf(q, 1.f / 13.f, 1.f / 11.f);
    r = fmaf(q, r, 1.f / 9.f);
    r = fmaf(q, r, 1.f / 7.f);
    r = fmaf(q, r, 1.f / 5.f);
    r = fmaf(q, r, 1.f / 3.f);
    r = fmaf(q, r, 1.f);
    r = fmaf(s + s, r, x > 0.f ? x : 0.f);
    return x == x ? r : x;
}

// Its values of a run of K positions from t, zeros from `end` on (which may lie before t).  VEC: rows and t are
// multiples of 16 bytes, so that a vector is inside the row of L positions or behind it.
template <typename T, int K, bool VEC>
__device__ __forceinline__ void load_run(const T *row, int t, int L, int end, float (&v)[K])
{
    if constexpr (VEC) {
        constexpr int E = 16 / (int)sizeof(T);
        static_assert(K % E == 0, "");
        #pragma unroll
        for (int i = 0; i < K; i += E) {
            Pack<T, E> x;
            if (t + i < end) x = *reinterpret_cast<const Pack<T, E> *>(row + t + i);
            #pragma unroll
            for (int j = 0; j < E; ++j) v[i + j] = t + i + j < end ? to_f(x.v[j]) : 0.f;
        }
    } else {
        #pragma unroll
        for (int i = 0; i < K; ++i) v[i] = t + i < end ? to_f(row[t + i]) : 0.f;
    }
}

template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int K, bool VEC>
__device__ __forceinline__ void store_run(T *row, int t, int L, const float (&v)[K])
{
    if constexpr (VEC) {
        constexpr int E = 16 / (int)sizeof(T);
        #pragma unroll
        for (int i = 0; i < K; i += E) {
            if (t + i >= L) continue;
            Pack<T, E> x;
            #pragma unroll
            for (int j = 0; j < E; ++j) x.v[j] = from_f<T>(v[i + j]);
            *reinterpret_cast<Pack<T, E> *>(row + t + i) = x;
        }
    } else {
        #pragma unroll
        for (int i = 0; i < K; ++i)
            if (t + i < L) row[t + i] = from_f<T>(v[i]);
    }
}

// Place of position t of a tile in a row of shared memory: four floats of gap after every 32, so that eight lanes
// eight positions apart read 16 bytes each without meeting in a bank.
__device__ __forceinline__ int spot(int t) { return t + ((t >> 5) << 2); }
constexpr int spots(int TT) { return TT + (TT / 32) * 4; }

// B or C of `count` states from s0 and TT positions from t0, in fp32, zeros from `end` on.
template <typename T, int TT, bool VEC>
__device__ __forceinline__ void stage_states(const T *base, int64_t L, int s0, int count, int t0, int end, float *sh)
{
    constexpr int E = VEC ? 16 / (int)sizeof(T) : 1;
    constexpr int PER = TT / E;
    for (int i = threadIdx.x; i < count * PER; i += blockDim.x) {
        const int s = i / PER, t = (i % PER) * E;
        float *to = sh + s * spots(TT) + spot(t);
        if constexpr (VEC) {
            Pack<T, E> x;
            if (t0 + t < end) x = *reinterpret_cast<const Pack<T, E> *>(base + (s0 + s) * L + t0 + t);
            #pragma unroll
            for (int j = 0; j < E; j += 4) {
                float4 f;
                f.x = t0 + t + j < end ? to_f(x.v[j]) : 0.f;
                f.y = t0 + t + j + 1 < end ? to_f(x.v[j + 1]) : 0.f;
                f.z = t0 + t + j + 2 < end ? to_f(x.v[j + 2]) : 0.f;
                f.w = t0 + t + j + 3 < end ? to_f(x.v[j + 3]) : 0.f;
                *reinterpret_cast<float4 *>(to + j) = f;
            }
        } else {
            *to = t0 + t < end ? to_f(base[(s0 + s) * L + t0 + t]) : 0.f;
        }
    }
}

template <int K>
__device__ __forceinline__ void read_run(const float *row, int t, float (&v)[K])
{
    #pragma unroll
    for (int i = 0; i < K; i += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(row + spot(t + i));
        v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
    }
}

// A log2 e, finite, so that a step of zero leaves a state as it was whatever A is.
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
