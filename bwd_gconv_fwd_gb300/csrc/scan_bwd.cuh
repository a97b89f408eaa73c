// scan_bwd.cuh -- gradients of the selective scan (see scan.cuh for the forward pass).
//
// With dy the gradient before the gate, w[t] what reaches h[t] from later positions and q[t] = exp(d[t] A) h[t-1]:
//   g[t] = C[t] dy[t] + w[t],   w[t-1] = exp(d[t] A) g[t]
//   dC[t] = sum_c dy h,   dB[t] = sum_c g d u,   du = d sum_s B g + D dy,   dd = u sum_s B g + sum_s A g q,
//   dA = sum_t d g q
// A tile's states are made again from the state that the forward pass kept before it, then the tile is walked
// backwards.  Sums over states stay in registers.  Sums over channels, which B and C share, are the costly ones: a
// thread adds its P channels in registers and then into a place of its own channel lane in shared memory; the warps of a
// block take different quarters of the states at a time, so that nothing is added by two of them at once and the order
// is fixed.
#pragma once

#include "scan.cuh"

namespace gconv {

template <typename T, int TL, int K, int P, bool VEC>
__global__ void __launch_bounds__(128) scan_bwd_kernel(const ScanArgs a)
{
    constexpr int CL = 32 / TL, TT = TL * K, ROW = spots(TT), OWN = CL * P;
    static_assert(TT % kScanMark == 0, "");
    extern __shared__ __align__(16) float smem[];
    const int warps = blockDim.x >> 5, CB = warps * OWN, all = CB * a.sets;
    float *sB = smem, *sC = sB + kScanStates * ROW, *accB = sC + kScanStates * ROW, *accC = accB + kScanStates * CL * ROW;
    float *sM = accC + kScanStates * CL * ROW;      // [CB][kScanStates]: states before the tile
    float *sA = sM + CB * kScanStates;              // [all][S]
    float *sdA = sA + all * a.S, *carry = sdA + all * a.S;        // [all][S], [2][all][S]
    float *sdD = carry + 2 * all * a.S, *sdb = sdD + all;         // [all]
    int64_t id = blockIdx.x;
    const int cb = (int)(id % a.ncb); id /= a.ncb;
    const int g = (int)(id % a.G); id /= a.G;
    const int chunk = (int)(id % a.chunks), n = (int)(id / a.chunks);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tl = lane % TL, cl = lane / TL;
    const int c0 = g * a.Cg + cb * all, left = min(all, a.Cg - cb * all);
    ptx::griddep_wait();
    const int end = sequence_end(a, n);
    for (int i = threadIdx.x; i < all * a.S; i += blockDim.x) {
        const int ch = i / a.S, s = i % a.S;
        sA[i] = ch < left ? decay_rate(a.A[(int64_t)c0 * a.S + i]) : 0.f;
        sdA[i] = 0.f;
        float w = 0.f;
        if (ch < left) {
            if (a.chunks > 1) w = a.init[(((int64_t)n * a.chunks + chunk) * a.S + s) * a.C + c0 + ch];
            else if (a.dstate_out) w = a.dstate_out[((int64_t)n * a.C + c0) * a.S + i];
        }
        carry[i] = w;
    }
    for (int i = threadIdx.x; i < all; i += blockDim.x) sdD[i] = sdb[i] = 0.f;
    const T *B = static_cast<const T *>(a.B) + n * a.sB + (int64_t)g * a.S * a.L;
    const T *Cm = static_cast<const T *>(a.Cm) + n * a.sC + (int64_t)g * a.S * a.L;
    const T *ub = static_cast<const T *>(a.u) + n * a.su, *db = static_cast<const T *>(a.delta) + n * a.sdelta;
    const T *yb = static_cast<const T *>(a.dy) + n * a.sdy;
    const T *zb = a.z ? static_cast<const T *>(a.z) + n * a.sz : nullptr;
    const T *pb = a.z ? static_cast<const T *>(a.pre) + (int64_t)n * a.C * a.L : nullptr;
    T *dub = static_cast<T *>(a.du) + n * a.sdu, *ddb = static_cast<T *>(a.ddelta) + n * a.sddelta;
    T *dzb = a.z ? static_cast<T *>(a.dz) + n * a.sdz : nullptr;
    float *part = a.ncb > 1 ? a.part + (((int64_t)n * a.G + g) * a.ncb + cb) * 2 * a.S * a.L : nullptr;
    int turn = 0;
    const int first = chunk * a.chunk_tiles, last = min(first + a.chunk_tiles, (a.L + TT - 1) / TT);
    for (int tile = last - 1; tile >= first; --tile) {
        const int t0 = tile * TT, t = t0 + tl * K;
        if (t0 >= end) {                            // behind the sequence: zeros (finish writes those of dB and dC from part)
            float zero[K];
            #pragma unroll
            for (int k = 0; k < K; ++k) zero[k] = 0.f;
            for (int ch = warp * CL + cl; ch < left; ch += warps * CL) {
                const int64_t row = (int64_t)(c0 + ch) * a.L;
                store_run<T, K, VEC>(dub + row, t, a.L, zero);
                store_run<T, K, VEC>(ddb + row, t, a.L, zero);
                if (dzb) store_run<T, K, VEC>(dzb + row, t, a.L, zero);
            }
            if (a.ncb == 1)
                for (int i = threadIdx.x; i < 2 * a.S * TT; i += blockDim.x) {
                    const int which = i / (a.S * TT), s = i / TT % a.S, at = t0 + i % TT;
                    T *to = static_cast<T *>(which ? a.dC : a.dB) + n * (which ? a.sdC : a.sdB);
                    if (at < a.L) to[((int64_t)g * a.S + s) * a.L + at] = from_f<T>(0.f);
                }
            continue;
        }
        const float *in = carry + turn * all * a.S;
        float *next = carry + (turn ^ 1) * all * a.S;
        for (int set = 0; set < a.sets; ++set) {
            const int mine = set * CB + warp * OWN + cl * P;
            float d[P][K], du[P][K], dy[P][K], sb[P][K], aq[P][K], sum[P];
            #pragma unroll
            for (int p = 0; p < P; ++p) {
                const int stop = mine + p < left ? end : 0;
                const int64_t row = (int64_t)(c0 + mine + p) * a.L;
                load_run<T, K, VEC>(ub + row, t, a.L, stop, du[p]);
                load_run<T, K, VEC>(db + row, t, a.L, stop, d[p]);
                load_run<T, K, VEC>(yb + row, t, a.L, stop, dy[p]);
                const float bias = a.bias && mine + p < left ? a.bias[c0 + mine + p] : 0.f;
                sum[p] = 0.f;
                #pragma unroll
                for (int k = 0; k < K; ++k) {
                    float v = d[p][k] + bias;
                    if (a.softplus) v = scan_softplus(v);
                    v = t + k < stop ? v : 0.f;
                    d[p][k] = v;
                    sum[p] += v;
                    du[p][k] *= v;
                    sb[p][k] = aq[p][k] = 0.f;
                }
                if (zb) {
                    float z[K];
                    load_run<T, K, VEC>(zb + row, t, a.L, stop, z);
                    #pragma unroll
                    for (int k = 0; k < K; ++k) dy[p][k] *= z[k] * scan_sigmoid(z[k]);
                    #pragma unroll
                    for (int k = 0; k < K; ++k) dy[p][k] = t + k < stop ? dy[p][k] : 0.f;
                }
            }
            for (int s0 = 0; s0 < a.S; s0 += kScanStates) {        // one round where there are several sets
                const int count = min(kScanStates, a.S - s0);
                if (set == 0) {
                    __syncthreads();                // the tile or states before are done with what is staged
                    stage_states<T, TT, VEC>(B, a.L, s0, count, t0, end, sB);
                    stage_states<T, TT, VEC>(Cm, a.L, s0, count, t0, end, sC);
                }
                __syncwarp();                       // the set before is done with sM
                for (int i = lane; i < OWN * count; i += 32) {
                    const int ch = warp * OWN + i % OWN, s = i / OWN;
                    sM[ch * kScanStates + s] = set * CB + ch < left
                        ? a.mark[(((int64_t)n * a.marks + t0 / kScanMark) * a.S + s0 + s) * a.C + c0 + set * CB + ch] : 0.f;
                }
                __syncwarp();
                if (set == 0) __syncthreads();
                const int per = (count + warps - 1) / warps;
                for (int round = 0; round < warps; ++round) {
                    const int from = (warp + round) % warps * per, to = min(count, from + per);
                    #pragma unroll 1
                    for (int s = from; s < to; ++s) {
                        float Bv[K], Cv[K], aB[K], aC[K];
                        read_run<K>(sB + s * ROW, tl * K, Bv);
                        read_run<K>(sC + s * ROW, tl * K, Cv);
                        #pragma unroll
                        for (int k = 0; k < K; ++k) aB[k] = aC[k] = 0.f;
                        #pragma unroll
                        for (int p = 0; p < P; ++p) {
                            const int at = (mine + p) * a.S + s0 + s;
                            const float rate = sA[at], cin = in[at];
                            const float before = sM[(warp * OWN + cl * P + p) * kScanStates + s];
                            float e[K], q[K], h = 0.f;
                            #pragma unroll
                            for (int k = 0; k < K; ++k) {
                                e[k] = ex2(d[p][k] * rate);
                                h = fmaf(e[k], h, du[p][k] * Bv[k]);
                            }
                            const float whole = ex2(sum[p] * rate);
                            float w = 0.f;
                            #pragma unroll
                            for (int k = K - 1; k >= 0; --k) w = e[k] * fmaf(Cv[k], dy[p][k], w);
                            float qh = whole, qw = whole;
                            if (tl == 0) h = fmaf(whole, before, h);
                            if (tl == TL - 1) w = fmaf(whole, cin, w);
                            #pragma unroll
                            for (int o = 1; o < TL; o <<= 1) {
                                const float hp = __shfl_up_sync(~0u, h, o, TL), qp = __shfl_up_sync(~0u, qh, o, TL);
                                const float wp = __shfl_down_sync(~0u, w, o, TL), rp = __shfl_down_sync(~0u, qw, o, TL);
                                if (tl >= o) { h = fmaf(qh, hp, h); qh *= qp; }
                                if (tl + o < TL) { w = fmaf(qw, wp, w); qw *= rp; }
                            }
                            if (tl == 0) next[at] = w;
                            h = __shfl_up_sync(~0u, h, 1, TL);
                            w = __shfl_down_sync(~0u, w, 1, TL);
                            if (tl == 0) h = before;
                            if (tl == TL - 1) w = cin;
                            #pragma unroll
                            for (int k = 0; k < K; ++k) {
                                q[k] = e[k] * h;
                                h = fmaf(du[p][k], Bv[k], q[k]);
                                aC[k] = fmaf(dy[p][k], h, aC[k]);
                            }
                            float dA = 0.f;
                            #pragma unroll
                            for (int k = K - 1; k >= 0; --k) {
                                const float gr = fmaf(Cv[k], dy[p][k], w);
                                aB[k] = fmaf(gr, du[p][k], aB[k]);
                                sb[p][k] = fmaf(gr, Bv[k], sb[p][k]);
                                const float x = gr * q[k];
                                aq[p][k] = fmaf(rate, x, aq[p][k]);
                                dA = fmaf(x, d[p][k], dA);
                                w = e[k] * gr;
                            }
                            #pragma unroll
                            for (int o = TL / 2; o > 0; o >>= 1) dA += __shfl_down_sync(~0u, dA, o, TL);
                            if (tl == 0) sdA[at] += dA;
                        }
                        float *toB = accB + (s * CL + cl) * ROW, *toC = accC + (s * CL + cl) * ROW;
                        #pragma unroll
                        for (int k = 0; k < K; k += 4) {
                            float4 *pB = reinterpret_cast<float4 *>(toB + spot(tl * K + k));
                            float4 *pC = reinterpret_cast<float4 *>(toC + spot(tl * K + k));
                            float4 vB = make_float4(aB[k], aB[k + 1], aB[k + 2], aB[k + 3]);
                            float4 vC = make_float4(aC[k], aC[k + 1], aC[k + 2], aC[k + 3]);
                            if (set | round) {
                                const float4 oB = *pB, oC = *pC;
                                vB.x += oB.x; vB.y += oB.y; vB.z += oB.z; vB.w += oB.w;
                                vC.x += oC.x; vC.y += oC.y; vC.z += oC.z; vC.w += oC.w;
                            }
                            *pB = vB;
                            *pC = vC;
                        }
                    }
                    __syncthreads();
                }
                if (set == a.sets - 1) {
                    for (int i = threadIdx.x; i < 2 * count * TT; i += blockDim.x) {
                        const int which = i / (count * TT), s = i / TT % count, at = i % TT;
                        const float *from = (which ? accC : accB) + s * CL * ROW + spot(at);
                        float v = 0.f;
                        #pragma unroll
                        for (int j = 0; j < CL; ++j) v += from[j * ROW];
                        if (t0 + at >= a.L) continue;
                        if (t0 + at >= end) v = 0.f;
                        if (part) {
                            part[((int64_t)which * a.S + s0 + s) * a.L + t0 + at] = v;
                        } else {
                            T *to = static_cast<T *>(which ? a.dC : a.dB) + n * (which ? a.sdC : a.sdB);
                            to[((int64_t)g * a.S + s0 + s) * a.L + t0 + at] = from_f<T>(v);
                        }
                    }
                }
            }
            #pragma unroll
            for (int p = 0; p < P; ++p) {
                const bool there = mine + p < left;
                const int64_t row = (int64_t)(c0 + mine + p) * a.L;
                const int stop = there ? end : 0;
                const float bias = a.bias && there ? a.bias[c0 + mine + p] : 0.f;
                const float skip = a.D && there ? a.D[c0 + mine + p] : 0.f;
                float v[K], dD = 0.f, dbias = 0.f;
                load_run<T, K, VEC>(ub + row, t, a.L, stop, v);
                #pragma unroll
                for (int k = 0; k < K; ++k) {
                    dD = fmaf(dy[p][k], v[k], dD);
                    aq[p][k] = fmaf(v[k], sb[p][k], aq[p][k] * kLn2);
                    du[p][k] = t + k < stop ? fmaf(d[p][k], sb[p][k], skip * dy[p][k]) : 0.f;
                }
                if (there) store_run<T, K, VEC>(dub + row, t, a.L, du[p]);
                if (a.softplus) {
                    load_run<T, K, VEC>(db + row, t, a.L, stop, v);
                    #pragma unroll
                    for (int k = 0; k < K; ++k) aq[p][k] *= scan_sigmoid(v[k] + bias);
                }
                #pragma unroll
                for (int k = 0; k < K; ++k) {
                    aq[p][k] = t + k < stop ? aq[p][k] : 0.f;
                    dbias += aq[p][k];
                }
                if (there) store_run<T, K, VEC>(ddb + row, t, a.L, aq[p]);
                if (zb) {
                    float z[K];
                    load_run<T, K, VEC>(zb + row, t, a.L, stop, z);
                    load_run<T, K, VEC>(pb + row, t, a.L, stop, v);
                    load_run<T, K, VEC>(yb + row, t, a.L, stop, du[p]);
                    #pragma unroll
                    for (int k = 0; k < K; ++k) {
                        const float sg = scan_sigmoid(z[k]);
                        v[k] = du[p][k] * v[k] * (sg * fmaf(z[k], 1.f - sg, 1.f));
                    }
                    #pragma unroll
                    for (int k = 0; k < K; ++k) v[k] = t + k < stop ? v[k] : 0.f;
                    if (there) store_run<T, K, VEC>(dzb + row, t, a.L, v);
                }
                #pragma unroll
                for (int o = TL / 2; o > 0; o >>= 1) {
                    dD += __shfl_down_sync(~0u, dD, o, TL);
                    dbias += __shfl_down_sync(~0u, dbias, o, TL);
                }
                if (tl == 0) { sdD[mine + p] += dD; sdb[mine + p] += dbias; }
            }
        }
        turn ^= 1;
    }
    __syncthreads();
    const float *fin = carry + turn * all * a.S;
    const int64_t base = ((int64_t)n * a.chunks + chunk) * a.C + c0;
    for (int i = threadIdx.x; i < left * a.S; i += blockDim.x) {
        a.pA[base * a.S + i] = sdA[i];
        if (a.dstate && chunk == 0) a.dstate[((int64_t)n * a.C + c0) * a.S + i] = fin[i];
    }
    for (int i = threadIdx.x; i < left; i += blockDim.x) {
        a.pD[base + i] = sdD[i];
        a.pb[base + i] = sdb[i];
    }
}

// What leaves a piece of a sequence backwards when nothing enters it, and its sum of d.
template <typename T, int TL, int K, int P, bool VEC>
__global__ void __launch_bounds__(128) scan_bwd_ends_kernel(const ScanArgs a)
{
    constexpr int CL = 32 / TL, TT = TL * K, ROW = spots(TT);
    extern __shared__ __align__(16) float smem[];
    const int warps = blockDim.x >> 5, CB = warps * CL * P;
    float *sC = smem, *sA = sC + kScanStates * ROW, *carry = sA + CB * a.S;
    int64_t id = blockIdx.x;
    const int blocks = (a.Cg + CB - 1) / CB;
    const int cb = (int)(id % blocks); id /= blocks;
    const int g = (int)(id % a.G); id /= a.G;
    const int chunk = (int)(id % a.chunks), n = (int)(id / a.chunks);
    const int lane = threadIdx.x & 31, tl = lane % TL;
    const int mine = ((threadIdx.x >> 5) * CL + lane / TL) * P;
    const int c0 = g * a.Cg + cb * CB, left = min(CB, a.Cg - cb * CB);
    ptx::griddep_wait();
    const int end = sequence_end(a, n);
    for (int i = threadIdx.x; i < CB * a.S; i += blockDim.x) {
        sA[i] = i / a.S < left ? decay_rate(a.A[(int64_t)c0 * a.S + i]) : 0.f;
        carry[i] = 0.f;
    }
    const T *Cm = static_cast<const T *>(a.Cm) + n * a.sC + (int64_t)g * a.S * a.L;
    float total[P];
    #pragma unroll
    for (int p = 0; p < P; ++p) total[p] = 0.f;
    int turn = 0;
    const int first = chunk * a.chunk_tiles, last = min(first + a.chunk_tiles, (a.L + TT - 1) / TT);
    for (int tile = last - 1; tile >= first; --tile) {
        const int t0 = tile * TT, t = t0 + tl * K;
        if (t0 >= end) continue;
        float d[P][K], dy[P][K], sum[P];
        #pragma unroll
        for (int p = 0; p < P; ++p) {
            const int stop = mine + p < left ? end : 0;
            const int64_t row = (int64_t)(c0 + mine + p) * a.L;
            load_run<T, K, VEC>(static_cast<const T *>(a.delta) + n * a.sdelta + row, t, a.L, stop, d[p]);
            load_run<T, K, VEC>(static_cast<const T *>(a.dy) + n * a.sdy + row, t, a.L, stop, dy[p]);
            const float bias = a.bias && mine + p < left ? a.bias[c0 + mine + p] : 0.f;
            sum[p] = 0.f;
            #pragma unroll
            for (int k = 0; k < K; ++k) {
                float v = d[p][k] + bias;
                if (a.softplus) v = scan_softplus(v);
                d[p][k] = t + k < stop ? v : 0.f;
                sum[p] += d[p][k];
            }
            total[p] += sum[p];
            if (a.z) {
                float z[K];
                load_run<T, K, VEC>(static_cast<const T *>(a.z) + n * a.sz + row, t, a.L, stop, z);
                #pragma unroll
                for (int k = 0; k < K; ++k) {
                    dy[p][k] *= z[k] * scan_sigmoid(z[k]);
                    dy[p][k] = t + k < stop ? dy[p][k] : 0.f;
                }
            }
        }
        const float *in = carry + turn * CB * a.S;
        float *next = carry + (turn ^ 1) * CB * a.S;
        for (int s0 = 0; s0 < a.S; s0 += kScanStates) {
            const int count = min(kScanStates, a.S - s0);
            __syncthreads();
            stage_states<T, TT, VEC>(Cm, a.L, s0, count, t0, end, sC);
            __syncthreads();
            #pragma unroll 1
            for (int s = 0; s < count; ++s) {
                float Cv[K];
                read_run<K>(sC + s * ROW, tl * K, Cv);
                #pragma unroll
                for (int p = 0; p < P; ++p) {
                    const int at = (mine + p) * a.S + s0 + s;
                    const float rate = sA[at];
                    float w = 0.f, qw = ex2(sum[p] * rate);
                    #pragma unroll
                    for (int k = K - 1; k >= 0; --k) w = ex2(d[p][k] * rate) * fmaf(Cv[k], dy[p][k], w);
                    if (tl == TL - 1) w = fmaf(qw, in[at], w);
                    #pragma unroll
                    for (int o = 1; o < TL; o <<= 1) {
                        const float wp = __shfl_down_sync(~0u, w, o, TL), rp = __shfl_down_sync(~0u, qw, o, TL);
                        if (tl + o < TL) { w = fmaf(qw, wp, w); qw *= rp; }
                    }
                    if (tl == 0) next[at] = w;
                }
            }
        }
        turn ^= 1;
    }
    __syncthreads();
    const float *fin = carry + turn * CB * a.S;
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
}

}  // namespace gconv
