// scan_ends.cuh -- the first of the two passes over a sequence that is cut in pieces (see scan.cuh): what leaves each piece when nothing
// enters it, forwards (the state) or backwards (what reaches the state before it), and the sum of d over it.
//
// Only a piece's end is wanted, not the states inside, so that no tile needs a scan: each of the eight lanes of a pair of channels
// walks over an eighth of the piece, eight positions a step, with its states in shared memory between the steps, and the eighths
// are joined once.  Both passes together, with the second pass's tiles of 64 neighbouring positions and a scan a tile here too,
// and this way: [1,2048,4096] 135 and 130 us forward, 311 and 308 backward; [1,256,65536] 247 and 237, 505 and 490.
#pragma once

#include "scan.cuh"

namespace gconv {

template <typename T, bool VEC, bool BACK>
__global__ void __launch_bounds__(128, 5) scan_ends_kernel(const __grid_constant__ ScanArgs a)
{
    constexpr int TL = kScanLanes, K = kScanRun, CL = 32 / TL, TT = kScanTile, ROW = spots(TT);
    extern __shared__ __align__(16) float smem[];
    const int pairs = (blockDim.x >> 5) * CL, CB = 2 * pairs, S = a.S, SP = S | 1;
    float *sB = smem, *sA = sB + kScanStates * ROW;               // B or C; rates [pairs][SP][2]
    float2 *held = reinterpret_cast<float2 *>(sA + CB * SP);      // [kScanStates][threads]
    int64_t id = blockIdx.x;
    const int blocks = (a.Cg - 1) / CB + 1;
    const int cb = (int)(id % blocks); id /= blocks;
    const int g = (int)(id % a.G); id /= a.G;
    const int chunk = (int)(id % a.chunks), n = (int)(id / a.chunks);
    const int lane = threadIdx.x & 31, tl = lane % TL;
    const int pair = (threadIdx.x >> 5) * CL + lane / TL, mine = 2 * pair;
    const int c0 = g * a.Cg + cb * CB, left = min(CB, a.Cg - cb * CB);
    ptx::griddep_wait();
    const int end = sequence_end(a, n);
    for (int i = threadIdx.x; i < CB * S; i += blockDim.x) {
        const int ch = i / S, s = i % S;
        sA[(ch >> 1) * 2 * SP + 2 * s + (ch & 1)] = ch < left && end > 0 ? decay_rate(a.A[(int64_t)c0 * S + i]) : 0.f;
    }
    const bool there0 = mine < left, there1 = mine + 1 < left;
    const int end0 = there0 ? end : 0, end1 = there1 ? end : 0;
    const int64_t row = ((int64_t)c0 + mine) * a.L;
    const T *from = static_cast<const T *>(BACK ? a.Cm : a.B) + n * (BACK ? a.sC : a.sB) + (int64_t)g * S * a.L;
    const T *db = static_cast<const T *>(a.delta) + n * a.sdelta;
    const T *xb = static_cast<const T *>(BACK ? a.dy : a.u) + n * (BACK ? a.sdy : a.su), *zb = static_cast<const T *>(a.z) + n * a.sz;
    const float2 bias = make_float2(a.bias && there0 ? a.bias[c0 + mine] : 0.f, a.bias && there1 ? a.bias[c0 + mine + 1] : 0.f);
    const float2 *rates = reinterpret_cast<const float2 *>(sA) + pair * SP;
    // the piece's positions, an eighth of them (whole runs) a lane; steps that lie behind the sequence in every lane are left out
    const int t0 = chunk * a.chunk_tiles * TT, each = a.chunk_tiles * K;
    const int steps = min(a.chunk_tiles, (max(0, min(end, a.L) - t0) + K - 1) / K);
    float2 total = both(0.f);
    for (int s0 = 0; s0 < S; s0 += kScanStates) {
        const int count = min(kScanStates, S - s0);
        for (int s = 0; s < count; ++s) held[s * blockDim.x + threadIdx.x] = both(0.f);
        for (int i = 0; i < steps; ++i) {
            const int step = (BACK ? steps - 1 - i : i) * K, t = t0 + tl * each + step;
            const Place<T, K, VEC> at(row, t, a.L, there0, there1);
            Run<T, K, VEC> rd, rx, rz;
            rd.load(db, at);
            rx.load(xb, at);
            if (BACK && a.z) rz.load(zb, at);
            States<T, VEC> f;
            f.load(from + (int64_t)s0 * a.L, a.L, count, t0 + step, each, end);
            float2 d[K], x[K], sum = both(0.f);
            #pragma unroll
            for (int k = 0; k < K; ++k) {
                d[k] = rd.at(k) + bias;
                if (a.softplus) d[k] = scan_softplus(d[k]);
                x[k] = rx.at(k);
                if (BACK && a.z) x[k] = x[k] * (rz.at(k) * scan_sigmoid(rz.at(k)));
            }
            clear_run<K>(t, end0, end1, d);
            clear_run<K>(t, end0, end1, x);
            #pragma unroll
            for (int k = 0; k < K; ++k) {
                sum = sum + d[k];
                if (!BACK) x[k] = x[k] * d[k];
            }
            if (s0 == 0) total = total + sum;
            __syncthreads();                        // the step before is done with sB
            f.store(from + (int64_t)s0 * a.L, a.L, count, t0 + step, each, end, sB);
            __syncthreads();
            const float *line = sB + spot(tl * K);
            float2 *h_ = held + threadIdx.x;
            #pragma unroll 2
            for (int s = 0; s < count; ++s, line += ROW, h_ += blockDim.x) {
                float Bv[K];
                read_run<K>(line, Bv);
                const float2 rate = rates[s0 + s];
                float2 h = *h_;
                if (!BACK) {
                    #pragma unroll
                    for (int k = 0; k < K; ++k) h = fma2(ex2(d[k] * rate), h, x[k] * both(Bv[k]));
                } else {
                    #pragma unroll
                    for (int k = K - 1; k >= 0; --k) h = ex2(d[k] * rate) * fma2(both(Bv[k]), x[k], h);
                }
                *h_ = h;
            }
        }
        if (steps == 0) __syncthreads();            // sA, where no step waited for it
        float *to = a.init + (((int64_t)n * a.chunks + chunk) * S + s0) * a.C + c0 + mine;
        for (int s = 0; s < count; ++s, to += a.C) {
            float2 h = held[s * blockDim.x + threadIdx.x], q = ex2(total * rates[s0 + s]);
            #pragma unroll
            for (int o = 1; o < TL; o <<= 1) {
                // this lane's positions, then those of the lane o further
                const float2 h1 = shift_down(h, o, TL), q1 = shift_down(q, o, TL);
                h = BACK ? fma2(q, h1, h) : fma2(q1, h, h1);
                q = q * q1;
            }
            if (tl == 0 && there0) to[0] = h.x;
            if (tl == 0 && there1) to[1] = h.y;
        }
    }
    #pragma unroll
    for (int o = TL / 2; o > 0; o >>= 1) total = total + shift_down(total, o, TL);
    float *to = a.dsum + ((int64_t)n * a.chunks + chunk) * a.C + c0 + mine;
    if (tl == 0 && there0) to[0] = total.x;
    if (tl == 0 && there1) to[1] = total.y;
}

}  // namespace gconv
