// scan_fwd.cuh -- the selective scan forward (see scan.cuh).
#pragma once

#include "scan.cuh"

namespace gconv {

// One block: W warps, each with CL = 32 / TL channel lanes of P channels, over the tiles of one piece of one sequence.
// ENDS: only what leaves the piece when zeros enter it, and the sum of d (the first of two passes over a long sequence).
template <typename T, int TL, int K, int P, bool VEC, bool ENDS>
__global__ void __launch_bounds__(128) scan_fwd_kernel(const ScanArgs a)
{
    constexpr int CL = 32 / TL, TT = TL * K;
    extern __shared__ __align__(16) float smem[];
    const int warps = blockDim.x >> 5, CB = warps * CL * P;
    float *sB = smem, *sC = sB + kScanStates * spots(TT), *sA = sC + (ENDS ? 0 : kScanStates * spots(TT));
    float *carry = sA + CB * a.S;                   // [2][CB][S]
    int64_t id = blockIdx.x;
    const int cb = (int)(id % a.ncb); id /= a.ncb;
    const int g = (int)(id % a.G); id /= a.G;
    const int chunk = (int)(id % a.chunks), n = (int)(id / a.chunks);
    const int lane = threadIdx.x & 31, tl = lane % TL;
    const int mine = ((threadIdx.x >> 5) * CL + lane / TL) * P;   // first of this thread's channels in the block
    const int c0 = g * a.Cg + cb * CB;                            // of the block
    const int left = min(CB, a.Cg - cb * CB);                     // channels of the block
    ptx::griddep_wait();
    const int end = sequence_end(a, n);
    for (int i = threadIdx.x; i < CB * a.S; i += blockDim.x) {
        const int ch = i / a.S, s = i % a.S;
        sA[i] = ch < left ? decay_rate(a.A[(int64_t)c0 * a.S + i]) : 0.f;
        float h = 0.f;
        if (ch < left && !ENDS) {
            if (a.chunks > 1) h = a.init[(((int64_t)n * a.chunks + chunk) * a.S + s) * a.C + c0 + ch];
            else if (a.state) h = a.state[((int64_t)n * a.C + c0) * a.S + i];
        }
        carry[i] = h;
    }
    const T *u = static_cast<const T *>(a.u) + n * a.su + (int64_t)(c0 + mine) * a.L;
    const T *dl = static_cast<const T *>(a.delta) + n * a.sdelta + (int64_t)(c0 + mine) * a.L;
    const T *z = a.z ? static_cast<const T *>(a.z) + n * a.sz + (int64_t)(c0 + mine) * a.L : nullptr;
    T *y = static_cast<T *>(a.y) + n * a.sy + (int64_t)(c0 + mine) * a.L;
    T *pre = a.pre ? static_cast<T *>(a.pre) + ((int64_t)n * a.C + c0 + mine) * a.L : nullptr;
    const T *B = static_cast<const T *>(a.B) + n * a.sB + (int64_t)g * a.S * a.L;
    const T *Cm = static_cast<const T *>(a.Cm) + n * a.sC + (int64_t)g * a.S * a.L;
    float bias[P], skip[P], total[P];
    #pragma unroll
    for (int p = 0; p < P; ++p) {
        bias[p] = a.bias && mine + p < left ? a.bias[c0 + mine + p] : 0.f;
        skip[p] = a.D && mine + p < left ? a.D[c0 + mine + p] : 0.f;
        total[p] = 0.f;
    }
    int turn = 0;
    const int tile_end = min((chunk + 1) * a.chunk_tiles, (a.L + TT - 1) / TT);
    for (int tile = chunk * a.chunk_tiles; tile < tile_end; ++tile) {
        const int t0 = tile * TT, t = t0 + tl * K;
        if (t0 >= end) {                            // behind the sequence: zeros, and the state stays
            if constexpr (!ENDS) {
                float zero[K];
                #pragma unroll
                for (int k = 0; k < K; ++k) zero[k] = 0.f;
                #pragma unroll
                for (int p = 0; p < P; ++p)
                    if (mine + p < left) store_run<T, K, VEC>(y + (int64_t)p * a.L, t, a.L, zero);
            }
            continue;
        }
        float d[P][K], du[P][K], out[P][K], sum[P];
        #pragma unroll
        for (int p = 0; p < P; ++p) {
            const int stop = mine + p < left ? end : 0;
            load_run<T, K, VEC>(u + (int64_t)p * a.L, t, a.L, stop, du[p]);
            load_run<T, K, VEC>(dl + (int64_t)p * a.L, t, a.L, stop, d[p]);
            sum[p] = 0.f;
            #pragma unroll
            for (int k = 0; k < K; ++k) {
                float v = d[p][k] + bias[p];
                if (a.softplus) v = scan_softplus(v);
                v = t + k < stop ? v : 0.f;
                d[p][k] = v;
                sum[p] += v;
                out[p][k] = skip[p] * du[p][k];
                du[p][k] *= v;
            }
            total[p] += sum[p];
        }
        for (int s0 = 0; s0 < a.S; s0 += kScanStates) {
            const int count = min(kScanStates, a.S - s0);
            __syncthreads();                        // the tile or states before are done with sB, sC and carry
            stage_states<T, TT, VEC>(B, a.L, s0, count, t0, end, sB);
            if constexpr (!ENDS) stage_states<T, TT, VEC>(Cm, a.L, s0, count, t0, end, sC);
            __syncthreads();
            const float *in = carry + turn * CB * a.S;
            float *next = carry + (turn ^ 1) * CB * a.S;
            #pragma unroll 1
            for (int s = 0; s < count; ++s) {
                float Bv[K], Cv[K];
                read_run<K>(sB + s * spots(TT), tl * K, Bv);
                if constexpr (!ENDS) read_run<K>(sC + s * spots(TT), tl * K, Cv);
                float e[P][K], h[P], q[P], cin[P];
                #pragma unroll
                for (int p = 0; p < P; ++p) {
                    const float rate = sA[(mine + p) * a.S + s0 + s];
                    cin[p] = in[(mine + p) * a.S + s0 + s];
                    h[p] = 0.f;
                    #pragma unroll
                    for (int k = 0; k < K; ++k) {
                        e[p][k] = ex2(d[p][k] * rate);
                        h[p] = fmaf(e[p][k], h[p], du[p][k] * Bv[k]);
                    }
                    q[p] = ex2(sum[p] * rate);
                    if (tl == 0) h[p] = fmaf(q[p], cin[p], h[p]);
                }
                #pragma unroll
                for (int o = 1; o < TL; o <<= 1) {
                    #pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const float hp = __shfl_up_sync(~0u, h[p], o, TL), qp = __shfl_up_sync(~0u, q[p], o, TL);
                        if (tl >= o) {
                            h[p] = fmaf(q[p], hp, h[p]);
                            q[p] *= qp;
                        }
                    }
                }
                #pragma unroll
                for (int p = 0; p < P; ++p) {
                    if (tl == TL - 1) next[(mine + p) * a.S + s0 + s] = h[p];
                    if constexpr (!ENDS) {
                        float v = __shfl_up_sync(~0u, h[p], 1, TL);
                        if (tl == 0) v = cin[p];
                        if (a.mark && t % kScanMark == 0 && t < a.L && mine + p < left)
                            a.mark[(((int64_t)n * a.marks + t / kScanMark) * a.S + s0 + s) * a.C + c0 + mine + p] = v;
                        #pragma unroll
                        for (int k = 0; k < K; ++k) {
                            v = fmaf(e[p][k], v, du[p][k] * Bv[k]);
                            out[p][k] = fmaf(Cv[k], v, out[p][k]);
                        }
                    }
                }
            }
        }
        turn ^= 1;
        if constexpr (!ENDS) {
            #pragma unroll
            for (int p = 0; p < P; ++p) {
                if (mine + p >= left) continue;
                if (z) {
                    float zv[K];
                    if (pre) store_run<T, K, VEC>(pre + (int64_t)p * a.L, t, a.L, out[p]);
                    load_run<T, K, VEC>(z + (int64_t)p * a.L, t, a.L, end, zv);
                    #pragma unroll
                    for (int k = 0; k < K; ++k) out[p][k] *= zv[k] * scan_sigmoid(zv[k]);
                }
                #pragma unroll
                for (int k = 0; k < K; ++k) out[p][k] = t + k < end ? out[p][k] : 0.f;
                store_run<T, K, VEC>(y + (int64_t)p * a.L, t, a.L, out[p]);
            }
        }
    }
    __syncthreads();
    const float *fin = carry + turn * CB * a.S;
    if constexpr (ENDS) {
        for (int i = threadIdx.x; i < left * a.S; i += blockDim.x) {
            const int s = i / left, ch = i % left;
            a.init[(((int64_t)n * a.chunks + chunk) * a.S + s) * a.C + c0 + ch] = fin[ch * a.S + s];
        }
        #pragma unroll
        for (int p = 0; p < P; ++p) {
            #pragma unroll
            for (int o = TL / 2; o > 0; o >>= 1) total[p] += __shfl_down_sync(~0u, total[p], o, TL);
            if (tl == 0 && mine + p < left) a.dsum[((int64_t)n * a.chunks + chunk) * a.C + c0 + mine + p] = total[p];
        }
    } else if (a.state_out && chunk == a.chunks - 1) {
        for (int i = threadIdx.x; i < left * a.S; i += blockDim.x) a.state_out[((int64_t)n * a.C + c0) * a.S + i] = fin[i];
    }
}

}  // namespace gconv
