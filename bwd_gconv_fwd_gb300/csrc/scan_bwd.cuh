// scan_bwd.cuh -- gradients of the selective scan (see scan.cuh for the forward pass).
//
// With dy the gradient before the gate and w[t] what reaches h[t] from later positions:
//   g[t] = C[t] dy[t] + w[t],   w[t-1] = exp(d[t] A) g[t]
//   dC[t] = sum_c dy h,   dB[t] = sum_c g d u,   du = d sum_s B g + D dy,   dd = u sum_s B g + sum_s A g q,
//   dA = sum_t d g q   (q[t] = exp(d[t] A) h[t-1])
// A tile's states are made again from the state that the forward pass kept before it, then the tile is walked
// backwards.  Sums over states stay in registers.  Sums over channels, which B and C share, are the costly ones: a
// thread adds its pair of channels and then into a place of its own channel lane in shared memory; the warps of a
// block take different quarters of the states at a time, so that nothing is added by two of them at once and the order
// is fixed.
//
// [8,2048,2048] bf16 with 16 states and a gate: 899 us, where bytes would take 78 and the fp32 pipe 270.  248 registers leave 8 warps
// an SM, whose waits for shuffles and shared memory bound it (issue slots 0.37, fp32 pipe 0.40, shared memory 0.34).  Rows off 16
// bytes sit at the limit of 255 and spill: 264 bytes stored and 152 read in fp32, 48 and 68 in bf16 with a gate, none without one.
#pragma once

#include "scan.cuh"

namespace gconv {

// SUMS: y before the gate is made again, for dz, one more multiply-add a state element (see scan_keeps; [8,2048,2048] bf16 899 us,
// 921 with the sums read from what the forward pass kept in bf16).
template <typename T, bool VEC, bool SUMS>
__global__ void __launch_bounds__(128, 2) scan_bwd_kernel(const __grid_constant__ ScanArgs a)
{
    constexpr int TL = kScanLanes, K = kScanRun, CL = 32 / TL, TT = kScanTile, ROW = spots(TT), OWN = kScanOwn;
    static_assert(TT % kScanMark == 0 && TL == 8, "a tile begins at a kept state; three steps a scan");
    const bool gated = scan_keeps<T> ? a.z != nullptr : SUMS;
    extern __shared__ __align__(16) float smem[];
    const int warps = blockDim.x >> 5, CB = warps * OWN, all = CB * a.sets, S = a.S, SP = S | 1;
    float *sB = smem, *sC = sB + kScanStates * ROW, *accB = sC + kScanStates * ROW, *accC = accB + kScanStates * CL * ROW;
    constexpr int MP = kScanStates + 1;             // SP and MP are odd, for the banks
    float *sM = accC + kScanStates * CL * ROW;      // [CB / 2][MP][2]: states before the tile
    float *sdA = sM + CB * MP;             // [warps][kScanStates][32][2]: the lanes' sums for dA
    float *sA = sdA + warps * kScanStates * 64;     // [all / 2][SP][2]
    float *accA = sA + all * SP, *carry = accA + all * SP;          // the same, [2] of the same
    float *sdD = carry + 2 * all * SP, *sdb = sdD + all, *sbias = sdb + all, *sskip = sbias + all;           // [all]
    int64_t id = blockIdx.x;
    const int cb = (int)(id % a.ncb); id /= a.ncb;
    const int g = (int)(id % a.G); id /= a.G;
    const int chunk = (int)(id % a.chunks), n = (int)(id / a.chunks);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tl = lane % TL, cl = lane / TL;
    const int c0 = g * a.Cg + cb * all, left = min(all, a.Cg - cb * all);
    ptx::griddep_wait();
    const int end = sequence_end(a, n);
    for (int i = threadIdx.x; i < all * S; i += blockDim.x) {
        const int ch = i / S, s = i % S, to = (ch >> 1) * 2 * SP + 2 * s + (ch & 1);
        sA[to] = ch < left && end > 0 ? decay_rate(a.A[(int64_t)c0 * S + i]) : 0.f;
        accA[to] = 0.f;
        float w = 0.f;
        if (ch < left) {
            if (a.chunks > 1) w = a.init[(((int64_t)n * a.chunks + chunk) * S + s) * a.C + c0 + ch];
            else if (a.dstate_out) w = a.dstate_out[((int64_t)n * a.C + c0) * S + i];
        }
        carry[to] = w;
    }
    for (int i = threadIdx.x; i < all; i += blockDim.x) {
        sdD[i] = sdb[i] = 0.f;
        sbias[i] = a.bias && i < left ? a.bias[c0 + i] : 0.f;
        sskip[i] = a.D && i < left ? a.D[c0 + i] : 0.f;
    }
    const T *B = static_cast<const T *>(a.B) + n * a.sB + (int64_t)g * S * a.L;
    const T *Cm = static_cast<const T *>(a.Cm) + n * a.sC + (int64_t)g * S * a.L;
    float *part = a.ncb > 1 ? a.part + (((int64_t)n * a.G + g) * a.ncb + cb) * 2 * S * a.L : nullptr;
    const int run = spot(tl * K);
    int turn = 0;
    const int first = chunk * a.chunk_tiles, last = min(first + a.chunk_tiles, (a.L + TT - 1) / TT);
    for (int tile = last - 1; tile >= first; --tile) {
        const int t0 = tile * TT, t = t0 + tl * K;
        if (t0 >= end) {                            // behind the sequence: zeros (scan_sum_kernel writes those of dB and dC from part)
            float2 zero[K];
            #pragma unroll
            for (int k = 0; k < K; ++k) zero[k] = both(0.f);
            for (int ch = 2 * (warp * CL + cl); ch < left; ch += CB) {
                const int64_t row = (int64_t)(c0 + ch) * a.L;
                const bool more = ch + 1 < left;
                store_run<T, K, VEC>(static_cast<T *>(a.du) + n * a.sdu + row, a.L, t, true, more, zero);
                store_run<T, K, VEC>(static_cast<T *>(a.ddelta) + n * a.sddelta + row, a.L, t, true, more, zero);
                if (gated) store_run<T, K, VEC>(static_cast<T *>(a.dz) + n * a.sdz + row, a.L, t, true, more, zero);
            }
            if (a.ncb == 1)
                for (int i = threadIdx.x; i < 2 * S * TT; i += blockDim.x) {
                    const int r = i / TT, which = r >= S, s = r - which * S, at = t0 + i % TT;
                    T *to = static_cast<T *>(which ? a.dC : a.dB) + n * (which ? a.sdC : a.sdB);
                    if (at < a.L) to[((int64_t)g * S + s) * a.L + at] = from_f<T>(0.f);
                }
            continue;
        }
        for (int set = 0; set < a.sets; ++set) {
            const int mine = set * CB + 2 * (warp * CL + cl), pair = mine >> 1;
            const bool there0 = mine < left, there1 = mine + 1 < left;
            const int end0 = there0 ? end : 0, end1 = there1 ? end : 0;
            const int64_t row = ((int64_t)c0 + mine) * a.L;
            const Place<T, K, VEC> at(row, t, a.L, there0, there1);
            const T *ub = static_cast<const T *>(a.u) + n * a.su, *db = static_cast<const T *>(a.delta) + n * a.sdelta;
            const T *yb = static_cast<const T *>(a.dy) + n * a.sdy, *zb = static_cast<const T *>(a.z) + n * a.sz;
            const float *pb = a.pre + (int64_t)n * a.C * a.L;
            Run<T, K, VEC> ru, rd, ry, rz;
            ru.load(ub, at);
            rd.load(db, at);
            ry.load(yb, at);
            if (gated) rz.load(zb, at);
            if (VEC && tile > first && t < a.L && there0) {        // the next tile's lines
                const int64_t o = at.x[0] - TT;
                fetch(ub + o);
                fetch(ub + o + at.step);
                fetch(db + o);
                fetch(db + o + at.step);
                fetch(yb + o);
                fetch(yb + o + at.step);
                if (gated) {
                    fetch(zb + o);
                    fetch(zb + o + at.step);
                    if (scan_keeps<T>) {
                        fetch(pb + o);
                        fetch(pb + o + at.step);
                    }
                }
            }
            States<T, VEC> fB, fC;
            constexpr int M = OWN * kScanStates / 32;
            float marks[M];
            auto ask = [&](int s0) {                // for what the next round of states needs from memory
                const int count = min(kScanStates, S - s0);
                if (set == 0) {
                    fB.load(B + (int64_t)s0 * a.L, a.L, count, t0, K, end);
                    fC.load(Cm + (int64_t)s0 * a.L, a.L, count, t0, K, end);
                }
                #pragma unroll
                for (int j = 0; j < M; ++j) {
                    const int i = lane + j * 32, s = i / OWN, at = set * CB + warp * OWN + i % OWN;
                    marks[j] = s < count && at < left
                        ? a.mark[(((int64_t)n * a.marks + t0 / kScanMark) * S + s0 + s) * a.C + c0 + at] : 0.f;
                }
            };
            ask(0);
            __syncthreads();                        // sbias, the first time; the tile or set before is done with what is staged
            float2 d[K], du[K], dy[K], sb[K], aq[K], pre[SUMS ? K : 1], sum = both(0.f);
            const float2 bias = *reinterpret_cast<const float2 *>(sbias + mine);
            #pragma unroll
            for (int k = 0; k < K; ++k) {
                d[k] = rd.at(k) + bias;
                if (a.softplus) d[k] = scan_softplus(d[k]);
                du[k] = ru.at(k);
                dy[k] = ry.at(k);
                if (gated) dy[k] = dy[k] * (rz.at(k) * scan_sigmoid(rz.at(k)));
            }
            clear_run<K>(t, end0, end1, d);
            clear_run<K>(t, end0, end1, du);
            clear_run<K>(t, end0, end1, dy);
            #pragma unroll
            for (int k = 0; k < K; ++k) {
                sum = sum + d[k];
                du[k] = du[k] * d[k];
                sb[k] = aq[k] = both(0.f);
                if (SUMS) pre[k] = both(0.f);
            }
            // steps of two and of four runs from here back and ahead: the scans' decays are exponentials of these instead of
            // more shuffles for every state (947 -> 928 us for [8,2048,2048])
            const float2 back2 = sum + shift_up(sum, 1, TL), back4 = back2 + shift_up(back2, 2, TL);
            const float2 next2 = sum + shift_down(sum, 1, TL), next4 = next2 + shift_down(next2, 2, TL);
            for (int s0 = 0; s0 < S; s0 += kScanStates) {          // one round where there are several sets
                const int count = min(kScanStates, S - s0);
                if (s0) {
                    ask(s0);
                    __syncthreads();
                }
                if (set == 0) {
                    fB.store(B + (int64_t)s0 * a.L, a.L, count, t0, K, end, sB);
                    fC.store(Cm + (int64_t)s0 * a.L, a.L, count, t0, K, end, sC);
                }
                #pragma unroll
                for (int j = 0; j < M; ++j) {
                    const int i = lane + j * 32, ch = i % OWN;
                    sM[((warp * CL + (ch >> 1)) * MP + i / OWN) * 2 + (ch & 1)] = marks[j];
                }
                __syncthreads();
                const int per = (count + warps - 1) / warps;
                const float2 *rates = reinterpret_cast<const float2 *>(sA) + pair * SP + s0;
                const float2 *in = reinterpret_cast<const float2 *>(carry + turn * all * SP) + pair * SP + s0;
                float2 *next = reinterpret_cast<float2 *>(carry + (turn ^ 1) * all * SP) + pair * SP + s0;
                const float2 *before = reinterpret_cast<const float2 *>(sM) + (warp * CL + cl) * MP;
                float2 *dAs = reinterpret_cast<float2 *>(sdA) + warp * kScanStates * 32;
                for (int round = 0; round < warps; ++round) {
                    const int begin = (warp + round) % warps * per, stop = min(count, begin + per);
                    const bool fresh = !(set | round);
                    const float *rowB = sB + begin * ROW + run, *rowC = sC + begin * ROW + run;
                    float *toB = accB + (begin * CL + cl) * ROW + run, *toC = accC + (begin * CL + cl) * ROW + run;
                    // two states side by side: a scan's shuffles wait less ([8,2048,2048] 986 -> 939 us)
                    #pragma unroll 2
                    for (int s = begin; s < stop; ++s, rowB += ROW, rowC += ROW, toB += CL * ROW, toC += CL * ROW) {
                        float Bv[K], Cv[K], aB[K], aC[K];
                        float2 e[K], q[K], h = both(0.f), w = both(0.f);
                        read_run<K>(rowB, Bv);
                        read_run<K>(rowC, Cv);
                        const float2 rate = rates[s], cin = in[s], hin = before[s];
                        #pragma unroll
                        for (int k = 0; k < K; ++k) {
                            e[k] = ex2(d[k] * rate);
                            h = fma2(e[k], h, du[k] * both(Bv[k]));
                        }
                        #pragma unroll
                        for (int k = K - 1; k >= 0; --k) w = e[k] * fma2(both(Cv[k]), dy[k], w);
                        float2 qh = ex2(sum * rate), qw = qh;
                        h = pick(tl == 0, fma2(qh, hin, h), h);
                        w = pick(tl == TL - 1, fma2(qw, cin, w), w);
                        #pragma unroll
                        for (int o = 1; o < TL; o <<= 1) {
                            // a lane below o (above TL - o) has runs in qh (qw) that are not there, and does not use it
                            h = pick(tl >= o, fma2(qh, shift_up(h, o, TL), h), h);
                            w = pick(tl + o < TL, fma2(qw, shift_down(w, o, TL), w), w);
                            if (2 * o < TL) {
                                qh = ex2((o == 1 ? back2 : back4) * rate);
                                qw = ex2((o == 1 ? next2 : next4) * rate);
                            }
                        }
                        if (tl == 0) next[s] = w;
                        h = pick(tl == 0, hin, shift_up(h, 1, TL));
                        w = pick(tl == TL - 1, cin, shift_down(w, 1, TL));
                        #pragma unroll
                        for (int k = 0; k < K; ++k) {
                            q[k] = e[k] * h;
                            h = fma2(du[k], both(Bv[k]), q[k]);
                            const float2 x = dy[k] * h;
                            aC[k] = x.x + x.y;
                            if (SUMS) pre[k] = fma2(both(Cv[k]), h, pre[k]);
                        }
                        float2 dA = both(0.f);
                        #pragma unroll
                        for (int k = K - 1; k >= 0; --k) {
                            const float2 gr = fma2(both(Cv[k]), dy[k], w), y = gr * du[k];
                            const float2 x = gr * q[k];
                            w = e[k] * gr;
                            aB[k] = y.x + y.y;
                            sb[k] = fma2(gr, both(Bv[k]), sb[k]);
                            aq[k] = fma2(rate, x, aq[k]);
                            dA = fma2(x, d[k], dA);
                        }
                        dAs[s * 32 + lane] = dA;
                        #pragma unroll
                        for (int k = 0; k < K; k += 4) {
                            float4 vB = make_float4(aB[k], aB[k + 1], aB[k + 2], aB[k + 3]);
                            float4 vC = make_float4(aC[k], aC[k + 1], aC[k + 2], aC[k + 3]);
                            if (!fresh) {
                                const float4 oB = *reinterpret_cast<const float4 *>(toB + k), oC = *reinterpret_cast<const float4 *>(toC + k);
                                vB.x += oB.x; vB.y += oB.y; vB.z += oB.z; vB.w += oB.w;
                                vC.x += oC.x; vC.y += oC.y; vC.z += oC.z; vC.w += oC.w;
                            }
                            *reinterpret_cast<float4 *>(toB + k) = vB;
                            *reinterpret_cast<float4 *>(toC + k) = vC;
                        }
                    }
                    __syncthreads();
                }
                ru.load(ub, at);                    // on their way during what follows (read after the last round of states)
                rd.load(db, at);
                // dA of the warp's channels: a lane adds the time lanes of its state and pair
                for (int i = lane; i < count * CL; i += 32) {
                    const int s = i / CL, j = i % CL;
                    float2 v = both(0.f);
                    #pragma unroll
                    for (int k = 0; k < TL; ++k) v = v + dAs[s * 32 + j * TL + (k + s) % TL];     // turned, for the banks
                    float2 *to = reinterpret_cast<float2 *>(accA) + ((set * CB + warp * OWN) / 2 + j) * SP + s0 + s;
                    *to = *to + v;
                }
                if (set == a.sets - 1) {
                    for (int i = threadIdx.x; i < 2 * count * (TT / 4); i += blockDim.x) {
                        const int r = i / (TT / 4), which = r >= count, s = r - which * count, at = i % (TT / 4) * 4;
                        const float *src = (which ? accC : accB) + s * CL * ROW + spot(at);
                        float4 v = *reinterpret_cast<const float4 *>(src);
                        #pragma unroll
                        for (int j = 1; j < CL; ++j) {
                            const float4 x = *reinterpret_cast<const float4 *>(src + j * ROW);
                            v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
                        }
                        const float o[4] = {v.x, v.y, v.z, v.w};
                        const int64_t line = ((int64_t)(part ? which : 0) * S + s0 + s) * a.L + t0 + at;
                        if (part && VEC) {
                            if (t0 + at < a.L) *reinterpret_cast<float4 *>(part + line) = v;
                        } else {
                            T *to = part ? nullptr : static_cast<T *>(which ? a.dC : a.dB) + n * (which ? a.sdC : a.sdB) + (int64_t)g * S * a.L;
                            #pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if (t0 + at + j >= a.L) continue;
                                if (part) part[line + j] = o[j];
                                else to[line + j] = from_f<T>(t0 + at + j < end ? o[j] : 0.f);
                            }
                        }
                    }
                }
            }
            const float2 skip = *reinterpret_cast<const float2 *>(sskip + mine);
            float2 dD = both(0.f), dbias = both(0.f);
            #pragma unroll
            for (int k = 0; k < K; ++k) {
                const float2 x = ru.at(k);
                if (SUMS) pre[k] = fma2(x, skip, pre[k]);
                aq[k] = fma2(x, sb[k], aq[k] * both(kLn2));
                if (a.softplus) aq[k] = aq[k] * scan_sigmoid(rd.at(k) + bias);
                sb[k] = fma2(d[k], sb[k], skip * dy[k]);
                dy[k] = dy[k] * x;
            }
            if (gated) {
                rz.load(zb, at);
                ry.load(yb, at);
                if constexpr (scan_keeps<T>) ru.load(pb, at);
            }
            clear_run<K>(t, end0, end1, aq);
            clear_run<K>(t, end0, end1, sb);
            clear_run<K>(t, end0, end1, dy);
            #pragma unroll
            for (int k = 0; k < K; ++k) {
                dbias = dbias + aq[k];
                dD = dD + dy[k];
            }
            store_run<T, K, VEC>(static_cast<T *>(a.du) + n * a.sdu + row, a.L, t, there0, there1, sb);
            store_run<T, K, VEC>(static_cast<T *>(a.ddelta) + n * a.sddelta + row, a.L, t, there0, there1, aq);
            if (gated) {
                #pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float2 z = rz.at(k), sg = scan_sigmoid(z);
                    const float2 rest = fma2(sg, both(-1.f), both(1.f));
                    sb[k] = ry.at(k) * (SUMS ? pre[SUMS ? k : 0] : ru.at(k)) * (sg * fma2(z, rest, both(1.f)));
                }
                clear_run<K>(t, end0, end1, sb);
                store_run<T, K, VEC>(static_cast<T *>(a.dz) + n * a.sdz + row, a.L, t, there0, there1, sb);
            }
            #pragma unroll
            for (int o = TL / 2; o > 0; o >>= 1) {
                dD = dD + shift_down(dD, o, TL);
                dbias = dbias + shift_down(dbias, o, TL);
            }
            if (tl == 0) {
                sdD[mine] += dD.x; sdD[mine + 1] += dD.y;
                sdb[mine] += dbias.x; sdb[mine + 1] += dbias.y;
            }
        }
        turn ^= 1;
    }
    __syncthreads();
    const float *fin = carry + turn * all * SP;
    const int64_t base = ((int64_t)n * a.chunks + chunk) * a.C + c0;
    for (int i = threadIdx.x; i < left * S; i += blockDim.x) {
        const int ch = i / S, s = i % S, from = (ch >> 1) * 2 * SP + 2 * s + (ch & 1);
        a.pA[base * S + i] = accA[from];
        if (a.dstate && chunk == 0) a.dstate[((int64_t)n * a.C + c0) * S + i] = fin[from];
    }
    for (int i = threadIdx.x; i < left; i += blockDim.x) {
        a.pD[base + i] = sdD[i];
        a.pb[base + i] = sdb[i];
    }
}

}  // namespace gconv
