// scan_fwd.cuh -- the selective scan forward (see scan.cuh).
//
// [8,2048,2048] bf16 with 16 states and a gate: 319 us (332 with what the gradient needs), where its four tensors would take 40 us at
// 6.8 TB/s, its exponentials 57 at 30 a clock and SM and the formula's four multiply-adds a state element 60 at 113 a clock and SM.
// 9.4 instructions a state element are issued, in 0.49 of the slots: the latency of shuffles and exponentials at 16 warps an SM.
#pragma once

#include "scan.cuh"

namespace gconv {

// One block: W warps, each with CL = 32 / TL lanes of a pair of channels, over the tiles of one piece of one sequence.
template <typename T, bool VEC>
__global__ void __launch_bounds__(128, 4) scan_fwd_kernel(const __grid_constant__ ScanArgs a)
{
    constexpr int TL = kScanLanes, K = kScanRun, CL = 32 / TL, TT = kScanTile, ROW = spots(TT);
    extern __shared__ __align__(16) float smem[];
    const int pairs = (blockDim.x >> 5) * CL, CB = 2 * pairs, S = a.S, SP = S | 1;
    float *sB = smem, *sC = sB + kScanStates * ROW, *sA = sC + kScanStates * ROW;    // sA: [pairs][SP][2]
    float *carry = sA + CB * SP;                    // [2][pairs][SP][2]; SP is odd, for the banks
    int64_t id = blockIdx.x;
    const int cb = (int)(id % a.ncb); id /= a.ncb;
    const int g = (int)(id % a.G); id /= a.G;
    const int chunk = (int)(id % a.chunks), n = (int)(id / a.chunks);
    const int lane = threadIdx.x & 31, tl = lane % TL;
    const int pair = (threadIdx.x >> 5) * CL + lane / TL, mine = 2 * pair;   // of the block's channels
    const int c0 = g * a.Cg + cb * CB;                            // of the block
    const int left = min(CB, a.Cg - cb * CB);                     // channels of the block
    ptx::griddep_wait();
    const int end = sequence_end(a, n);
    for (int i = threadIdx.x; i < CB * S; i += blockDim.x) {
        const int ch = i / S, s = i % S, to = (ch >> 1) * 2 * SP + 2 * s + (ch & 1);
        sA[to] = ch < left && end > 0 ? decay_rate(a.A[(int64_t)c0 * S + i]) : 0.f;
        float h = 0.f;
        if (ch < left) {
            if (a.chunks > 1) h = a.init[(((int64_t)n * a.chunks + chunk) * S + s) * a.C + c0 + ch];
            else if (a.state) h = a.state[((int64_t)n * a.C + c0) * S + i];
        }
        carry[to] = h;
    }
    const bool there0 = mine < left, there1 = mine + 1 < left;
    const int end0 = there0 ? end : 0, end1 = there1 ? end : 0;
    const int64_t row = ((int64_t)c0 + mine) * a.L;
    const T *u = static_cast<const T *>(a.u) + n * a.su;
    const T *Cm = static_cast<const T *>(a.Cm) + n * a.sC + (int64_t)g * S * a.L;
    const float2 bias = make_float2(a.bias && there0 ? a.bias[c0 + mine] : 0.f, a.bias && there1 ? a.bias[c0 + mine + 1] : 0.f);
    const float2 skip = make_float2(a.D && there0 ? a.D[c0 + mine] : 0.f, a.D && there1 ? a.D[c0 + mine + 1] : 0.f);
    const int run = spot(tl * K);
    int turn = 0;
    const int tile_end = min((chunk + 1) * a.chunk_tiles, (a.L + TT - 1) / TT);
    for (int tile = chunk * a.chunk_tiles; tile < tile_end; ++tile) {
        const int t0 = tile * TT, t = t0 + tl * K;
        if (t0 >= end) {                            // behind the sequence: zeros, and the state stays
            float2 zero[K];
            #pragma unroll
            for (int k = 0; k < K; ++k) zero[k] = both(0.f);
            store_run<T, K, VEC>(static_cast<T *>(a.y) + n * a.sy + row, a.L, t, there0, there1, zero);
            continue;
        }
        const T *dl = static_cast<const T *>(a.delta) + n * a.sdelta;
        const T *B = static_cast<const T *>(a.B) + n * a.sB + (int64_t)g * S * a.L;
        const Place<T, K, VEC> at(row, t, a.L, there0, there1);
        Run<T, K, VEC> ru, rd;
        ru.load(u, at);
        rd.load(dl, at);
        if (VEC && t + TT < end0) {                 // the next tile's lines, and what is read after the states
            if (a.z) {
                const T *z = static_cast<const T *>(a.z) + n * a.sz + at.x[0];
                fetch(z);
                fetch(z + at.step);
            }
            if (tile + 1 < tile_end) {
                fetch(u + at.x[0] + TT);
                fetch(u + at.x[0] + TT + at.step);
                fetch(dl + at.x[0] + TT);
                fetch(dl + at.x[0] + TT + at.step);
            }
        }
        States<T, VEC> fB, fC;
        fB.load(B, a.L, min(kScanStates, S), t0, K, end);
        fC.load(Cm, a.L, min(kScanStates, S), t0, K, end);
        float2 d[K], du[K], out[K], sum = both(0.f);
        #pragma unroll
        for (int k = 0; k < K; ++k) {
            d[k] = rd.at(k) + bias;
            if (a.softplus) d[k] = scan_softplus(d[k]);
            du[k] = ru.at(k);
        }
        clear_run<K>(t, end0, end1, d);
        clear_run<K>(t, end0, end1, du);
        #pragma unroll
        for (int k = 0; k < K; ++k) {
            sum = sum + d[k];
            out[k] = du[k] * skip;
            du[k] = du[k] * d[k];
        }
        const bool marks = a.mark && t % kScanMark == 0 && t < a.L;
        float *mark = marks ? a.mark + (((int64_t)n * a.marks + t / kScanMark) * S) * a.C + c0 + mine : nullptr;
        for (int s0 = 0; s0 < S; s0 += kScanStates) {
            const int count = min(kScanStates, S - s0);
            if (s0) {
                fB.load(B + (int64_t)s0 * a.L, a.L, count, t0, K, end);
                fC.load(Cm + (int64_t)s0 * a.L, a.L, count, t0, K, end);
            }
            __syncthreads();                        // the tile or states before are done with sB, sC and carry
            fB.store(B + (int64_t)s0 * a.L, a.L, count, t0, K, end, sB);
            fC.store(Cm + (int64_t)s0 * a.L, a.L, count, t0, K, end, sC);
            __syncthreads();
            const float2 *rates = reinterpret_cast<const float2 *>(sA) + pair * SP + s0;
            const float2 *in = reinterpret_cast<const float2 *>(carry + turn * CB * SP) + pair * SP + s0;
            float2 *next = reinterpret_cast<float2 *>(carry + (turn ^ 1) * CB * SP) + pair * SP + s0;
            const float *rowB = sB + run, *rowC = sC + run;
            // two states side by side: a scan's shuffles wait less ([8,2048,2048] 375 -> 340 us)
            #pragma unroll 2
            for (int s = 0; s < count; ++s, rowB += ROW, rowC += ROW, mark += a.C) {
                float Bv[K];
                float2 e[K], h = both(0.f);
                read_run<K>(rowB, Bv);
                const float2 rate = rates[s], cin = in[s];
                #pragma unroll
                for (int k = 0; k < K; ++k) {
                    e[k] = ex2(d[k] * rate);
                    h = fma2(e[k], h, du[k] * both(Bv[k]));
                }
                float2 q = ex2(sum * rate);
                h = pick(tl == 0, fma2(q, cin, h), h);
                #pragma unroll
                for (int o = 1; o < TL; o <<= 1) {
                    // q of a lane below 2 o is not read again, so that only what goes into h is held back
                    h = pick(tl >= o, fma2(q, shift_up(h, o, TL), h), h);
                    if (2 * o < TL) q = q * shift_up(q, o, TL);
                }
                if (tl == TL - 1) next[s] = h;
                float2 v = pick(tl == 0, cin, shift_up(h, 1, TL));
                if (marks) {
                    if (there0) mark[0] = v.x;
                    if (there1) mark[1] = v.y;
                }
                float Cv[K];
                read_run<K>(rowC, Cv);
                #pragma unroll
                for (int k = 0; k < K; ++k) {
                    v = fma2(e[k], v, du[k] * both(Bv[k]));
                    out[k] = fma2(both(Cv[k]), v, out[k]);
                }
            }
        }
        turn ^= 1;
        if (a.z) {
            Run<T, K, VEC> rz;
            rz.load(static_cast<const T *>(a.z) + n * a.sz, at);
            if constexpr (scan_keeps<T>) {
                if (a.pre) store_run<T, K, VEC>(a.pre + (int64_t)n * a.C * a.L + row, a.L, t, there0, there1, out);
            }
            #pragma unroll
            for (int k = 0; k < K; ++k) out[k] = out[k] * (rz.at(k) * scan_sigmoid(rz.at(k)));
        }
        clear_run<K>(t, end0, end1, out);
        store_run<T, K, VEC>(static_cast<T *>(a.y) + n * a.sy + row, a.L, t, there0, there1, out);
    }
    __syncthreads();
    const float *fin = carry + turn * CB * SP;
    if (a.state_out && chunk == a.chunks - 1) {
        for (int i = threadIdx.x; i < left * S; i += blockDim.x) {
            const int ch = i / S, s = i % S;
            a.state_out[((int64_t)n * a.C + c0) * S + i] = fin[(ch >> 1) * 2 * SP + 2 * s + (ch & 1)];
        }
    }
}

}  // namespace gconv
