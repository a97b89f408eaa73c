// scan.cu -- extern "C" entry points of the selective scan: checks, launch shapes, and the kernels around the scans
// (short sequences, the join of a sequence's pieces, the gradients' sums over blocks).
#include "scan_internal.h"

#include <algorithm>
#include <climits>

namespace gconv {

namespace {

// Positions of the short form; sequences a thread of it.  [64,2048,L] bf16, 16 states and a gate: 8 positions 24 us, 76 as a tile
// of which seven eighths are empty; 9 as a tile 90.  With room for sixteen positions a thread 9 take 38 us and 16 52 (76), but 2
// take 32 for 20 and 8 36 for 24.
constexpr int kTokenMost = 8, kTokenMany = 2;

// ---- short sequences ----------------------------------------------------------------
//
// What a single new position has to move is its state, 8 bytes a state and channel.  Four lanes share a channel, four
// neighbouring states each (one 16-byte access where FOUR: states in fours, on 16 bytes), so that a warp's accesses are
// whole lines; sums over states are two shuffles.  NB: sequences a thread takes, all of whose states are on their way
// before the first is used; the channel's rates are read once for them.  [64,2048,1], 16 states: 6.9 us in a graph (2.6 by its bytes).
template <typename T, int LT, int NB, bool FOUR>
__global__ void __launch_bounds__(128, LT > 1 ? 4 : NB > 1 ? 8 : 10) scan_token_kernel(const __grid_constant__ ScanArgs a)
{
    const unsigned ng = blockIdx.x / (unsigned)a.ncb, cb = blockIdx.x - ng * a.ncb;
    const int n0 = (int)(ng / (unsigned)a.G) * NB, g = (int)(ng % (unsigned)a.G);
    const int q = threadIdx.x & 3, ch = (int)cb * 32 + (threadIdx.x >> 2);
    const bool there = ch < a.Cg;
    const int c = g * a.Cg + (there ? ch : 0), S = a.S;
    ptx::griddep_wait();
    // the last block's missing sequences stand for the first one of it, and are not written
    int n[NB], end[NB];
    #pragma unroll
    for (int i = 0; i < NB; ++i) {
        n[i] = n0 + i < a.N ? n0 + i : n0;
        end[i] = sequence_end(a, n[i]);
    }
    const float *rates = a.A + (int64_t)c * S;
    Pack<float, 4> h[NB], rate;
    Pack<T, 4> Bv[NB], Cv[NB];          // of the one position (LT 1)
    auto load = [&](int s0) {
        const int s = s0 + 4 * q;
        const Pack<float, 4> none{};
        if constexpr (FOUR) {
            rate = s < S ? *reinterpret_cast<const Pack<float, 4> *>(rates + s) : none;
            #pragma unroll
            for (int i = 0; i < NB; ++i)
                h[i] = s < S && a.state ? *reinterpret_cast<const Pack<float, 4> *>(a.state + ((int64_t)n[i] * a.C + c) * S + s) : none;
        } else {
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                rate.v[j] = s + j < S ? rates[s + j] : 0.f;
                #pragma unroll
                for (int i = 0; i < NB; ++i) h[i].v[j] = s + j < S && a.state ? a.state[((int64_t)n[i] * a.C + c) * S + s + j] : 0.f;
            }
        }
        if constexpr (LT == 1) {
            #pragma unroll
            for (int i = 0; i < NB; ++i) {
                const T *B = static_cast<const T *>(a.B) + n[i] * a.sB + g * S + s;
                const T *Cm = static_cast<const T *>(a.Cm) + n[i] * a.sC + g * S + s;
                Bv[i] = Cv[i] = Pack<T, 4>{};
                if constexpr (FOUR) {
                    if (s < S) {
                        Bv[i] = *reinterpret_cast<const Pack<T, 4> *>(B);
                        Cv[i] = *reinterpret_cast<const Pack<T, 4> *>(Cm);
                    }
                } else {
                    #pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (s + j < S) {
                            Bv[i].v[j] = B[j];
                            Cv[i].v[j] = Cm[j];
                        }
                }
            }
        }
    };
    load(0);
    const float bias = a.bias ? a.bias[c] : 0.f, skip = a.D ? a.D[c] : 0.f;
    float d[NB][LT], du[NB][LT], out[NB][LT], z[NB][LT];
    #pragma unroll
    for (int i = 0; i < NB; ++i) {
        const T *dl = static_cast<const T *>(a.delta) + n[i] * a.sdelta + (int64_t)c * a.L;
        const T *u = static_cast<const T *>(a.u) + n[i] * a.su + (int64_t)c * a.L;
        const T *zr = static_cast<const T *>(a.z) + n[i] * a.sz + (int64_t)c * a.L;
        #pragma unroll
        for (int t = 0; t < LT; ++t) {
            d[i][t] = t < end[i] ? to_f(dl[t]) : 0.f;
            du[i][t] = t < end[i] ? to_f(u[t]) : 0.f;
            z[i][t] = a.z && t < end[i] ? to_f(zr[t]) : 0.f;
        }
    }
    #pragma unroll
    for (int i = 0; i < NB; ++i) {
        #pragma unroll
        for (int t = 0; t < LT; ++t) {
            float v = d[i][t] + bias;
            if (a.softplus) v = scan_softplus(v);
            d[i][t] = t < end[i] ? v : 0.f;
            out[i][t] = q == 0 ? skip * du[i][t] : 0.f;
            du[i][t] *= d[i][t];
        }
    }
    for (int s0 = 0; s0 < S; s0 += 16) {
        const int s = s0 + 4 * q;
        if (s0) load(s0);
        #pragma unroll
        for (int i = 0; i < NB; ++i) {
            const bool real = there && n0 + i < a.N;
            const T *B = static_cast<const T *>(a.B) + n[i] * a.sB + ((int64_t)g * S + s) * a.L;
            const T *Cm = static_cast<const T *>(a.Cm) + n[i] * a.sC + ((int64_t)g * S + s) * a.L;
            const int64_t at = ((int64_t)n[i] * a.C + c) * S + s;
            Pack<float, 4> now = h[i];
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (s + j >= S) continue;
                const float r = decay_rate(rate.v[j]);
                float v = h[i].v[j];
                if (a.mark && real) a.mark[((int64_t)n[i] * S + s + j) * a.C + c] = v;
                #pragma unroll
                for (int t = 0; t < LT; ++t) {
                    if (t >= end[i]) continue;
                    v = fmaf(ex2(d[i][t] * r), v, du[i][t] * to_f(LT == 1 ? Bv[i].v[j] : B[(int64_t)j * a.L + t]));
                    out[i][t] = fmaf(to_f(LT == 1 ? Cv[i].v[j] : Cm[(int64_t)j * a.L + t]), v, out[i][t]);
                }
                now.v[j] = v;
            }
            if (!a.state_out || !real) continue;
            if constexpr (FOUR) {
                if (s < S) *reinterpret_cast<Pack<float, 4> *>(a.state_out + at) = now;
            } else {
                #pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (s + j < S) a.state_out[at + j] = now.v[j];
            }
        }
    }
    #pragma unroll
    for (int i = 0; i < NB; ++i) {
        #pragma unroll
        for (int t = 0; t < LT; ++t) {
            out[i][t] += __shfl_xor_sync(~0u, out[i][t], 1);
            out[i][t] += __shfl_xor_sync(~0u, out[i][t], 2);
            if (((LT > 1 ? t : i) & 3) != q || t >= a.L || !there || n0 + i >= a.N) continue;
            const int64_t row = (int64_t)c * a.L + t;
            float v = out[i][t];
            if (a.z) {
                if (scan_keeps<T> && a.pre && t < end[i]) a.pre[(int64_t)n[i] * a.C * a.L + row] = v;
                v *= z[i][t] * scan_sigmoid(z[i][t]);
            }
            static_cast<T *>(a.y)[n[i] * a.sy + row] = from_f<T>(t < end[i] ? v : 0.f);
        }
    }
}

// What enters each piece of a sequence, in place of what leaves it when nothing enters, backwards for the gradient.  A column of
// threads has a state of a channel: each joins a run of pieces (read before any is written), the column's runs are joined
// through shared memory, and every thread goes over its run again from what enters that.  Latencies bound it: with one
// thread for all pieces, sixteen read at a time, the whole call took 225 us for [1,256,65536] (147 pieces), 211 so; sixteen
// pieces a run are no faster.
constexpr int kScanJoin = 8, kScanColumn = 8;       // pieces of a run, threads of a column

__global__ void __launch_bounds__(32 * kScanColumn) scan_join_kernel(const __grid_constant__ ScanArgs a, int back)
{
    __shared__ float value[kScanColumn][32], total[kScanColumn][32];
    const int x = threadIdx.x & 31, r = threadIdx.x >> 5, rows = blockDim.x >> 5;
    const int64_t at = (int64_t)blockIdx.x * 32 + x, sc = (int64_t)a.S * a.C;
    const bool on = at < a.N * sc;
    const int64_t i = on ? at : 0;
    const int n = (int)(i / sc), s = (int)(i % sc / a.C), c = (int)(i % a.C);
    ptx::griddep_wait();
    const float rate = sequence_end(a, n) > 0 ? decay_rate(a.A[(int64_t)c * a.S + s]) : 0.f;
    const float *first = back ? a.dstate_out : a.state;
    float h = first ? first[((int64_t)n * a.C + c) * a.S + s] : 0.f;
    const int64_t step = back ? -1 : 1, begin = (int64_t)n * a.chunks + (back ? a.chunks - 1 : 0);
    float *to = a.init + begin * sc + (int64_t)s * a.C + c;
    const float *sum = a.dsum + begin * a.C + c;
    for (int k0 = 0; k0 < a.chunks; k0 += rows * kScanJoin) {
        const int k1 = k0 + r * kScanJoin;
        float left[kScanJoin], d[kScanJoin];
        #pragma unroll
        for (int k = 0; k < kScanJoin; ++k) {
            const bool there = on && k1 + k < a.chunks;
            left[k] = there ? to[(k1 + k) * step * sc] : 0.f;
            d[k] = there ? sum[(k1 + k) * step * a.C] : 0.f;
        }
        float v = 0.f, all = 0.f;
        #pragma unroll
        for (int k = 0; k < kScanJoin; ++k) {
            all += d[k];
            d[k] = ex2(d[k] * rate);
            v = fmaf(d[k], v, left[k]);
        }
        value[r][x] = v;
        total[r][x] = all;
        __syncthreads();
        float in = h;
        for (int q = 0; q < rows; ++q) {
            if (q == r) in = h;
            h = fmaf(ex2(total[q][x] * rate), h, value[q][x]);
        }
        __syncthreads();
        #pragma unroll
        for (int k = 0; k < kScanJoin; ++k) {
            if (on && k1 + k < a.chunks) to[(k1 + k) * step * sc] = in;
            in = fmaf(d[k], in, left[k]);
        }
    }
}

// ---- sums over the gradient's blocks ------------------------------------------------

struct SumArgs {
    const float *part, *pA, *pD, *pb;
    int N, G, ncb, S, C, L, rows;       // rows: of pA, pD and pb
    unsigned blocks;                    // that add dB and dC; the rest add the parameters' gradients
    void *dB, *dC;
    int64_t sdB, sdC;
    float *dA, *dD, *db;
    const int *lengths;
};

template <typename T, int V>
__global__ void __launch_bounds__(256) scan_sum_kernel(const SumArgs a)
{
    ptx::griddep_wait();
    if (blockIdx.x < a.blocks) {
        const int64_t SL = (int64_t)a.S * a.L, per = SL / V;
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
        if (i >= (int64_t)a.N * a.G * 2 * per) return;
        const int64_t e = i % per * V;
        const int which = (int)(i / per % 2);
        const int64_t ng = i / per / 2;
        const int n = (int)(ng / a.G), g = (int)(ng % a.G);
        int end = a.L;
        if (a.lengths) end = min(max(a.lengths[n], 0), a.L);
        const int t = (int)(e % a.L);
        Pack<float, V> v{};
        bool any = false;
        #pragma unroll
        for (int j = 0; j < V; ++j) any |= (V == 1 ? t : (int)((e + j) % a.L)) < end;
        if (any) {
            const float *p = a.part + (ng * a.ncb * 2 + which) * SL + e;
            #pragma unroll 8
            for (int b = 0; b < a.ncb; ++b) {
                const Pack<float, V> x = *reinterpret_cast<const Pack<float, V> *>(p + (int64_t)b * 2 * SL);
                #pragma unroll
                for (int j = 0; j < V; ++j) v.v[j] += x.v[j];
            }
        }
        Pack<T, V> o;
        #pragma unroll
        for (int j = 0; j < V; ++j) o.v[j] = static_cast<T>((V == 1 ? t : (int)((e + j) % a.L)) < end ? v.v[j] : 0.f);
        T *to = static_cast<T *>(which ? a.dC : a.dB) + n * (which ? a.sdC : a.sdB) + g * SL + e;
        *reinterpret_cast<Pack<T, V> *>(to) = o;
        return;
    }
    // 32 columns a block, eight threads a column
    __shared__ float sh[8][32];
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t CS = (int64_t)a.C * a.S, col = (int64_t)(blockIdx.x - a.blocks) * 32 + lane;
    const float *p = nullptr;
    float *to = nullptr;
    int64_t step = a.C;
    if (col < CS) { p = a.pA + col; to = a.dA + col; step = CS; }
    else if (col < CS + a.C) { p = a.pD + (col - CS); to = a.dD ? a.dD + (col - CS) : nullptr; }
    else if (col < CS + 2 * a.C) { p = a.pb + (col - CS - a.C); to = a.db ? a.db + (col - CS - a.C) : nullptr; }
    float v = 0.f;
    if (to)
        for (int r = k; r < a.rows; r += 8) v += p[r * step];
    sh[k][lane] = v;
    __syncthreads();
    if (k == 0 && to) {
        #pragma unroll
        for (int j = 1; j < 8; ++j) v += sh[j][lane];
        *to = v;
    }
}

// ---- checks and shapes ----------------------------------------------------------------

int esize(gconv_dtype dt) { return dt == GCONV_BF16 ? 2 : 4; }

bool check_scan(const gconv_scan *s, gconv_dtype dt)
{
    if (!s || (dt != GCONV_F32 && dt != GCONV_BF16)) return false;
    if (s->N < 0 || s->C < 1 || s->L < 1 || s->L > (1 << 30) || s->groups < 1 || s->C % s->groups) return false;
    if (s->states < 1 || s->states > kScanMaxStates || s->softplus < 0 || s->softplus > 1) return false;
    const int64_t CL = (int64_t)s->C * s->L, GSL = (int64_t)s->groups * s->states * s->L;
    // 2^40 elements a tensor, which also keeps every product below 64 bits
    if (std::max(CL, GSL) > ((int64_t)1 << 40) / std::max(1, s->N) || (int64_t)s->C * s->states > INT_MAX) return false;
    for (long long b : {s->u_batch, s->delta_batch, s->z_batch, s->y_batch, s->dy_batch, s->du_batch, s->ddelta_batch, s->dz_batch})
        if (b != 0 && (b < CL || b > ((int64_t)1 << 40))) return false;
    for (long long b : {s->B_batch, s->C_batch, s->dB_batch, s->dC_batch})
        if (b != 0 && (b < GSL || b > ((int64_t)1 << 40))) return false;
    return true;
}

int64_t marks_of(const gconv_scan &s) { return (s.L + kScanMark - 1) / kScanMark; }

size_t up16(size_t v) { return (v + 15) / 16 * 16; }

size_t saved_marks(const gconv_scan &s) { return up16((size_t)s.N * marks_of(s) * s.states * s.C * sizeof(float)); }

struct ScanPlan {
    ScanShape shape, ends;
    int token;
    int ncb, sets, chunks, chunk_tiles;
    size_t o_init, o_dsum, o_part, o_pA, o_pD, o_pb, bytes;
};

// Time of a launch, in units of a tile of one block alone on an SM.  A tile's time with k blocks on each SM counts as 1, 1.2,
// 1.4, 1.6 (forward; 7.5 us with 16 states alone, 12 us four at a time) or 1, 1.5 (gradient; 13 and 17 us, two fit) and a
// block's start as a quarter tile.  These and the factors of a cut were fitted together to the times of ten shapes at some
// twenty cuts each: what they pick is 0.3% (forward) and 2.5% (gradient) above the best of those, 2 and 12% at worst.
double scan_cost(bool back, int64_t blocks, double tiles)
{
    tiles += 0.25;
    const int most = back ? 2 : 4;
    const double more = back ? 0.5 : 0.2;
    const int64_t slots = (int64_t)num_sms() * most, last = blocks % slots;
    return tiles * (blocks / slots * (1 + more * (most - 1)) + (last ? 1 + more * ((last + num_sms() - 1) / num_sms() - 1) : 0));
}

bool plan_scan(const gconv_scan &s, bool back, ScanPlan *p)
{
    *p = ScanPlan{};
    const int Cg = s.C / s.groups, S = s.states;
    p->sets = p->chunks = 1;
    if (!back && s.L <= kTokenMost) {
        p->token = 1;
        p->ncb = (Cg - 1) / 32 + 1;
        // two sequences a thread once the blocks of one go round more than once: [64,2048,1], 16 states 6.9 us, 7.5 with
        // one a thread and 8.1 with four
        int64_t grid = (int64_t)s.N * s.groups * p->ncb;
        p->token = s.L == 1 && grid > (int64_t)num_sms() * 10 ? kTokenMany : 1;
        grid = (int64_t)((s.N + p->token - 1) / p->token) * s.groups * p->ncb;
        p->shape.grid = (unsigned)grid;
        return grid <= INT_MAX;
    }
    const int own = kScanOwn, CL = 32 / kScanLanes, TT = kScanTile;
    const int units = (Cg - 1) / own + 1, tiles = (s.L + TT - 1) / TT;      // a warp's channels, tiles of a sequence
    // Warps a block, channel sets that a block of the gradient takes in turn (fewer partial sums of dB and dC; where B and C
    // of all the states fit), and pieces that a sequence is cut into: the cheapest.  A cut takes a pass over the
    // pieces before (0.3 of the forward pass, 0.15 of the gradient) and two launches.  Measured in us, uncut and cut:
    // forward [1,2048,4096] 370 and 112 (16 pieces), [1,256,65536] 5997 and 205 (147), [8,2048,2048] 319 and 409 (8);
    // gradient [1,2048,4096] 687 and 275 (32), [8,2048,2048] 919, 898 in two sets, 962 in 8 pieces.
    double best = 0;
    int warps = 1;
    for (int sets = 1; sets <= (back && S <= kScanStates ? 2 : 1); ++sets) {
        const int ncb = (units + 4 * sets - 1) / (4 * sets), w = (units + ncb * sets - 1) / (ncb * sets);
        const int64_t blocks = (int64_t)s.N * s.groups * ncb;
        for (int chunks = 1; chunks <= tiles; chunks = std::max(chunks + 1, std::min(chunks + chunks / 8, tiles))) {
            const int each = (tiles + chunks - 1) / chunks, real = (tiles + each - 1) / each;
            double cost = scan_cost(back, blocks * real, (double)each * sets);
            if (real > 1) cost = cost * (back ? 1.15 : 1.3) + 1.0;
            if (sets == 1) cost *= 1.02;             // twice the partial sums
            if (best == 0 || cost < best) {
                best = cost;
                warps = w; p->sets = sets; p->ncb = ncb; p->chunks = real; p->chunk_tiles = each;
            }
            if (blocks * real > (int64_t)num_sms() * 64) break;
        }
    }
    const int per = warps * own * p->sets;
    const int64_t grid = (int64_t)s.N * s.groups * p->ncb * p->chunks;
    const int64_t ends_grid = back ? (int64_t)s.N * s.groups * ((Cg - 1) / (warps * own) + 1) * p->chunks : grid;
    if (grid > INT_MAX || ends_grid > INT_MAX) return false;
    if (p->chunks > 1 && (int64_t)s.N * S > ((int64_t)INT_MAX * 32 - 31) / s.C) return false;        // scan_join_kernel's blocks
    const int row = spots(TT);
    const int SP = S | 1;
    auto floats = [&](bool ends) -> size_t {
        if (ends) return (size_t)kScanStates * row + (size_t)warps * (own * SP + 64 * kScanStates);
        if (!back) return (size_t)2 * kScanStates * row + 3 * (size_t)warps * own * SP;
        return (size_t)(2 + 2 * CL) * kScanStates * row + (size_t)warps * (own * (kScanStates + 1) + 64 * kScanStates) +
               4 * (size_t)per * SP + 4 * per;
    };
    p->shape = {warps, 0, (unsigned)grid, floats(false) * 4};
    p->ends = {warps, 0, (unsigned)ends_grid, floats(true) * 4};
    size_t at = 0;
    auto take = [&](size_t n) { const size_t was = at; at += up16(n * sizeof(float)); return was; };
    const size_t pieces = (size_t)s.N * p->chunks;
    if (p->chunks > 1) {
        p->o_init = take(pieces * S * s.C);
        p->o_dsum = take(pieces * s.C);
    }
    if (back) {
        if (p->ncb > 1) p->o_part = take((size_t)s.N * s.groups * p->ncb * 2 * S * s.L);
        p->o_pA = take(pieces * s.C * S);
        p->o_pD = take(pieces * s.C);
        p->o_pb = take(pieces * s.C);
    }
    p->bytes = at;
    return true;
}

void scan_args(const gconv_scan &s, const ScanPlan &p, void *ws, ScanArgs *a)
{
    a->N = s.N; a->C = s.C; a->L = s.L; a->G = s.groups; a->S = s.states; a->Cg = s.C / s.groups;
    a->softplus = s.softplus;
    a->ncb = p.ncb; a->sets = p.sets; a->chunks = p.chunks; a->chunk_tiles = p.chunk_tiles;
    a->marks = (int)marks_of(s);
    const int64_t CL = (int64_t)s.C * s.L, GSL = (int64_t)s.groups * s.states * s.L;
    auto step = [](long long b, int64_t dense) { return b ? (int64_t)b : dense; };
    a->su = step(s.u_batch, CL); a->sdelta = step(s.delta_batch, CL); a->sz = step(s.z_batch, CL); a->sy = step(s.y_batch, CL);
    a->sB = step(s.B_batch, GSL); a->sC = step(s.C_batch, GSL);
    a->sdy = step(s.dy_batch, CL); a->sdu = step(s.du_batch, CL); a->sddelta = step(s.ddelta_batch, CL);
    a->sdz = step(s.dz_batch, CL); a->sdB = step(s.dB_batch, GSL); a->sdC = step(s.dC_batch, GSL);
    char *w = static_cast<char *>(ws);
    a->init = reinterpret_cast<float *>(w + p.o_init);
    a->dsum = reinterpret_cast<float *>(w + p.o_dsum);
    a->part = reinterpret_cast<float *>(w + p.o_part);
    a->pA = reinterpret_cast<float *>(w + p.o_pA);
    a->pD = reinterpret_cast<float *>(w + p.o_pD);
    a->pb = reinterpret_cast<float *>(w + p.o_pb);
}

bool on(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Rows that 16-byte vectors cover: L, the steps between sequences and the addresses are multiples of 16 bytes.
struct Rows { const void *p; int64_t step; };
bool vectors(const gconv_scan &s, gconv_dtype dt, std::initializer_list<Rows> rows)
{
    const int E = 16 / esize(dt);
    if (s.L % E) return false;
    for (const Rows &r : rows)
        if (!on(r.p, 16) || (s.N > 1 && r.step % E)) return false;
    return true;
}

void join(const ScanArgs &a, int back, cudaStream_t st)
{
    const int rows = std::min((a.chunks + kScanJoin - 1) / kScanJoin, kScanColumn);
    launch_dependent(scan_join_kernel, (unsigned)(((int64_t)a.N * a.S * a.C + 31) / 32), 32u * rows, 0, st, a, back);
}

gconv_status done() { return cudaGetLastError() == cudaSuccess ? GCONV_OK : GCONV_ERR_CUDA; }

}  // namespace

}  // namespace gconv

using namespace gconv;

extern "C" {

size_t gconv_scan_saved_size(const gconv_scan *scan, gconv_dtype dtype, int gated)
{
    if (!check_scan(scan, dtype)) return (size_t)-1;
    return saved_marks(*scan) + (gated ? (size_t)scan->N * scan->C * scan->L * esize(dtype) : 0);
}

size_t gconv_scan_workspace_size(const gconv_scan *scan, gconv_dtype dtype, int backward)
{
    ScanPlan p;
    if (!check_scan(scan, dtype) || !plan_scan(*scan, backward != 0, &p)) return (size_t)-1;
    return scan->N ? p.bytes : 0;
}

gconv_status gconv_scan_fwd(const gconv_scan *scan, gconv_dtype dtype, const void *u, const void *delta, const float *A,
                            const void *B, const void *C, const float *D, const void *z, const float *delta_bias,
                            const float *state, const int *lengths, void *y, float *state_out, void *saved, void *workspace,
                            size_t workspace_bytes, void *stream)
{
    ScanPlan p;
    if (!check_scan(scan, dtype) || !plan_scan(*scan, false, &p)) return GCONV_ERR_INVALID_ARG;
    if (scan->N == 0) return GCONV_OK;
    if (!u || !delta || !A || !B || !C || !y) return GCONV_ERR_INVALID_ARG;
    for (const void *q : {u, delta, B, C, z, (const void *)y})
        if (!on(q, esize(dtype))) return GCONV_ERR_INVALID_ARG;
    for (const void *q : {(const void *)A, (const void *)D, (const void *)delta_bias, (const void *)state, (const void *)lengths,
                          (const void *)state_out})
        if (!on(q, 4)) return GCONV_ERR_INVALID_ARG;
    if (!on(saved, 16)) return GCONV_ERR_INVALID_ARG;
    if (p.bytes && (!workspace || workspace_bytes < p.bytes || !on(workspace, 16))) return GCONV_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    ScanArgs a{};
    scan_args(*scan, p, workspace, &a);
    a.u = u; a.delta = delta; a.A = A; a.B = B; a.Cm = C; a.D = D; a.z = z; a.bias = delta_bias; a.state = state;
    a.lengths = lengths; a.y = y; a.state_out = state_out;
    a.mark = static_cast<float *>(saved);
    a.pre = saved && z && dtype == GCONV_F32 ? a.mark + saved_marks(*scan) / sizeof(float) : nullptr;
    if (p.token) {
        const bool four = scan->states % 4 == 0 && on(A, 16) && on(state, 16) && on(state_out, 16) && on(B, 4 * esize(dtype)) &&
                          on(C, 4 * esize(dtype)) && (scan->N == 1 || (a.sB % 4 == 0 && a.sC % 4 == 0));
        using H = __nv_bfloat16;
        auto pick = [&](auto few, auto one, auto many) { return scan->L > 1 ? few : p.token == 1 ? one : many; };
        constexpr int M = kTokenMost, K = kTokenMany;
        auto *kernel = dtype == GCONV_BF16
            ? (four ? pick(scan_token_kernel<H, M, 1, true>, scan_token_kernel<H, 1, 1, true>, scan_token_kernel<H, 1, K, true>)
                    : pick(scan_token_kernel<H, M, 1, false>, scan_token_kernel<H, 1, 1, false>, scan_token_kernel<H, 1, K, false>))
            : (four ? pick(scan_token_kernel<float, M, 1, true>, scan_token_kernel<float, 1, 1, true>, scan_token_kernel<float, 1, K, true>)
                    : pick(scan_token_kernel<float, M, 1, false>, scan_token_kernel<float, 1, 1, false>, scan_token_kernel<float, 1, K, false>));
        launch_dependent(kernel, p.shape.grid, 128u, 0, st, a);
        return done();
    }
    p.shape.vec = p.ends.vec = vectors(*scan, dtype, {{u, a.su}, {delta, a.sdelta}, {z, a.sz}, {B, a.sB}, {C, a.sC}, {y, a.sy},
                                                      {a.pre, (int64_t)scan->C * scan->L}});
    auto *start = dtype == GCONV_BF16 ? scan_fwd_bf16 : scan_fwd_f32;
    if (p.chunks > 1) {
        start(p.ends, true, a, st);
        join(a, 0, st);
    }
    start(p.shape, false, a, st);
    return done();
}

gconv_status gconv_scan_bwd(const gconv_scan *scan, gconv_dtype dtype, const void *u, const void *delta, const float *A,
                            const void *B, const void *C, const float *D, const void *z, const float *delta_bias,
                            const int *lengths, const void *saved, const void *dy, const float *dstate_out, void *du,
                            void *ddelta, float *dA, void *dB, void *dC, float *dD, void *dz, float *ddelta_bias, float *dstate,
                            void *workspace, size_t workspace_bytes, void *stream)
{
    ScanPlan p;
    if (!check_scan(scan, dtype) || !plan_scan(*scan, true, &p)) return GCONV_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((z == nullptr) != (dz == nullptr) || !A || !dA || !on(dA, 4) || !on(dD, 4) || !on(ddelta_bias, 4)) return GCONV_ERR_INVALID_ARG;
    if (scan->N == 0) {
        const size_t c = (size_t)scan->C * sizeof(float);
        if (cudaMemsetAsync(dA, 0, c * scan->states, st) != cudaSuccess || (dD && cudaMemsetAsync(dD, 0, c, st) != cudaSuccess) ||
            (ddelta_bias && cudaMemsetAsync(ddelta_bias, 0, c, st) != cudaSuccess))
            return GCONV_ERR_CUDA;
        return GCONV_OK;
    }
    if (!u || !delta || !B || !C || !saved || !dy || !du || !ddelta || !dB || !dC) return GCONV_ERR_INVALID_ARG;
    for (const void *q : {u, delta, B, C, z, dy, (const void *)du, (const void *)ddelta, (const void *)dB, (const void *)dC,
                          (const void *)dz})
        if (!on(q, esize(dtype))) return GCONV_ERR_INVALID_ARG;
    for (const void *q : {(const void *)A, (const void *)D, (const void *)delta_bias, (const void *)lengths, (const void *)dstate_out,
                          (const void *)dstate})
        if (!on(q, 4)) return GCONV_ERR_INVALID_ARG;
    if (!on(saved, 16)) return GCONV_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < p.bytes || !on(workspace, 16)) return GCONV_ERR_WORKSPACE;
    ScanArgs a{};
    scan_args(*scan, p, workspace, &a);
    a.u = u; a.delta = delta; a.A = A; a.B = B; a.Cm = C; a.D = D; a.z = z; a.bias = delta_bias; a.lengths = lengths;
    a.mark = const_cast<float *>(static_cast<const float *>(saved));
    a.pre = z && dtype == GCONV_F32 ? a.mark + saved_marks(*scan) / sizeof(float) : nullptr;
    a.dy = dy; a.dstate_out = dstate_out; a.du = du; a.ddelta = ddelta; a.dB = dB; a.dC = dC; a.dz = dz; a.dstate = dstate;
    p.shape.vec = p.ends.vec = vectors(*scan, dtype, {{u, a.su}, {delta, a.sdelta}, {z, a.sz}, {B, a.sB}, {C, a.sC}, {dy, a.sdy},
                                                      {du, a.sdu}, {ddelta, a.sddelta}, {dz, a.sdz},
                                                      {a.pre, (int64_t)scan->C * scan->L}});
    auto *start = dtype == GCONV_BF16 ? scan_bwd_bf16 : scan_bwd_f32;
    if (p.chunks > 1) {
        start(p.ends, true, a, st);
        join(a, 1, st);
    }
    start(p.shape, false, a, st);
    SumArgs f{};
    f.part = a.part; f.pA = a.pA; f.pD = a.pD; f.pb = a.pb;
    f.N = a.N; f.G = a.G; f.ncb = p.ncb; f.S = a.S; f.C = a.C; f.L = a.L; f.rows = a.N * p.chunks;
    f.dB = dB; f.dC = dC; f.sdB = a.sdB; f.sdC = a.sdC; f.dA = dA; f.dD = dD; f.db = ddelta_bias; f.lengths = lengths;
    const size_t v4 = 4 * esize(dtype);
    const bool four = (int64_t)a.S * a.L % 4 == 0 && on(dB, v4) && on(dC, v4) && (a.N == 1 || (a.sdB % 4 == 0 && a.sdC % 4 == 0));
    if (p.ncb > 1) {
        const int64_t items = (int64_t)a.N * a.G * 2 * a.S * a.L / (four ? 4 : 1);
        if ((items + 255) / 256 > INT_MAX) return GCONV_ERR_INVALID_ARG;
        f.blocks = (unsigned)((items + 255) / 256);
    }
    const unsigned grid = f.blocks + (unsigned)(((int64_t)a.C * (a.S + 2) + 31) / 32);
    auto *sum = dtype == GCONV_BF16 ? (four ? scan_sum_kernel<__nv_bfloat16, 4> : scan_sum_kernel<__nv_bfloat16, 1>)
                                    : (four ? scan_sum_kernel<float, 4> : scan_sum_kernel<float, 1>);
    launch_dependent(sum, grid, 256u, 0, st, f);
    return done();
}

}  // extern "C"
