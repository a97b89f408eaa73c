// causal.cu -- short causal convolution along the positions of each channel, and its gradients.
//
//   v[t] = bias + sum_k w[k] x[t - K + 1 + k],   y = act(v),   x before position 0 from the state
//   dv = dy act'(v),   dx[t] = sum_k w[k] dv[t + K - 1 - k],   dw[k] = sum dv[t] x[t - K + 1 + k],   db = sum dv
//
// Two or three tensors go through once, at 2 K + 8 operations an element (6 K + 12 for the gradients); with what it takes to
// unpack, shift and round them issue slots bound it (0.62 of the launch) beside memory (4.2 TB/s, 32 us for [8,2048,2048] bf16, 4 taps).
// Accesses are 16 bytes where the tensors' rows begin at the same place of 16 bytes (element by element otherwise).  A lane takes the elements of one row (channel of a sequence) that lie in one or two
// neighbouring 16-byte pieces of memory, so rows of odd length, which begin anywhere, are read in whole pieces too; only a row's
// two ends go element by element.  What the window needs from the piece before is read again (from L1).
// TX lanes (a power of two, a warp where rows are long) are a worker: it keeps a channel's weights, and its sums for their
// gradients, over its share of the sequences and their pieces.
#include "scan.cuh"

#include <algorithm>
#include <climits>

namespace gconv {

namespace {

constexpr int kCausalMost = 8;          // taps
// Positions of the form with one thread a row, for one new position of a sequence and few more.  [64,2048,L] bf16, 4 taps: 4
// positions 2.1 us, 8.5 by workers; 5 by workers 11.1.  With room for sixteen a thread 5 take 2.6, 8 4.7 (15 by workers), 16 14
// (27, in fp32 12 and 5.4), so that the border could lie at 8.
constexpr int kCausalShort = 4;
constexpr int kCausalThreads = 128;
constexpr int kCausalBack = 8;          // elements a lane of the gradient

struct CausalArgs {
    int N, C, L, act;
    int TX, segs, splits;               // lanes of a worker, pieces of a row, workers that share a channel
    const void *x, *y, *dy;
    int64_t sx, sy, sdy, sdx;
    const float *w, *bias;
    const void *state;
    void *state_out;
    const int *lengths;
    void *out;                          // y or dx
    const void *dstate_out;
    void *dstate;
    float *part;                        // [splits][C][K + 1]
};

__host__ __device__ __forceinline__ int causal_end(const CausalArgs &a, int n)
{
    if (!a.lengths) return a.L;
    const int v = a.lengths[n];
    return v < 0 ? 0 : v < a.L ? v : a.L;
}

// Elements t .. t + M - 1 of a row, zeros outside [0, end): the slow way, for a row's ends.
template <typename T, int M>
__device__ __forceinline__ void load_some(const T *row, int t, int end, float *v)
{
    #pragma unroll
    for (int j = 0; j < M; ++j) v[j] = t + j >= 0 && t + j < end ? to_f(row[t + j]) : 0.f;
}

// Elements t .. t + M - 1 to a row of L; `whole`: all of them are in it, and the address is on 16 bytes.
template <typename T, int M, bool VEC>
__device__ __forceinline__ void store_pieces(T *row, int t, int L, bool whole, const float (&v)[M])
{
    constexpr int V = 16 / (int)sizeof(T);
    if (VEC && whole) {
        #pragma unroll
        for (int i = 0; i < M; i += V) {
            Pack<T, V> x;
            #pragma unroll
            for (int j = 0; j < V; j += 2) put2(x.v + j, v[i + j], v[i + j + 1]);
            *reinterpret_cast<Pack<T, V> *>(row + t + i) = x;
        }
    } else {
        #pragma unroll
        for (int j = 0; j < M; ++j)
            if (t + j >= 0 && t + j < L) row[t + j] = from_f<T>(v[j]);
    }
}

// win[i]: x at t - H + i for i < H + M (zeros outside the sequence, the state before it); d, unless `other` is null: another
// tensor's M elements from t.  `whole`: the run is inside the sequence or behind it, and begins the row or has whole pieces
// before it.  What it has not is then read from `safe`, the row's first place on 16 bytes, so that no load needs a
// condition and all are on their way before the first is used; a lane behind the sequence gets values that are not its own.
template <typename T, int M, int H, bool VEC>
__device__ __forceinline__ void load_window(const T *row, const T *state, int t, int end, bool whole, int safe, float (&win)[H + M],
                                            const T *other, float (&d)[M])
{
    constexpr int V = 16 / (int)sizeof(T), BACK = (H + V - 1) / V;      // pieces before t
    if (VEC && whole) {
        const int from = t < end ? t : safe, before = from >= BACK * V ? from - BACK * V : safe;
        Pack<T, V> p[BACK ? BACK : 1], x[M / V], o[M / V];
        #pragma unroll
        for (int i = 0; i < M / V; ++i) x[i] = *reinterpret_cast<const Pack<T, V> *>(row + from + i * V);
        #pragma unroll
        for (int i = 0; i < BACK; ++i) p[i] = *reinterpret_cast<const Pack<T, V> *>(row + before + i * V);
        if (other) {
            #pragma unroll
            for (int i = 0; i < M / V; ++i) o[i] = *reinterpret_cast<const Pack<T, V> *>(other + from + i * V);
        }
        #pragma unroll
        for (int i = 0; i < H; ++i) win[i] = t ? to_f(p[(BACK * V - H + i) / V].v[(BACK * V - H + i) % V]) : 0.f;
        #pragma unroll
        for (int i = 0; i < M; ++i) win[H + i] = to_f(x[i / V].v[i % V]);
        if (other) {
            #pragma unroll
            for (int i = 0; i < M; ++i) d[i] = to_f(o[i / V].v[i % V]);
        }
        return;
    }
    load_some<T, H + M>(row, t - H, end, win);
    if (other) load_some<T, M>(other, t, end, d);
    if (state && t < H) {
        #pragma unroll
        for (int i = 0; i < H + M; ++i) {
            const int at = t - H + i;
            if (at < 0 && at >= -H) win[i] = to_f(state[H + at]);
        }
    }
}

// Whether a run of M elements from t takes the short way through load_window and the stores.
template <typename T, int M, int H>
__device__ __forceinline__ bool whole_run(int t, int end, int L, bool state)
{
    constexpr int V = 16 / (int)sizeof(T), BACK = (H + V - 1) / V;
    if (end < M + V) return t >= L;              // `safe` and a run from there are in the sequence
    if (t >= end) return t >= L || t + M <= L;
    return t + M <= end && (t >= BACK * V || (t == 0 && !state));
}

template <typename T>
__device__ __forceinline__ int phase_of(const T *row)
{
    return (int)((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % (16 / sizeof(T)));
}

template <typename T>
__device__ __forceinline__ int first_place(int phase) { return phase ? 16 / (int)sizeof(T) - phase : 0; }

// The worker that a thread belongs to.  There may be 2^36 threads, but no more than 2^32 workers (TX divides a block).
__host__ __device__ __forceinline__ unsigned worker_of(unsigned block, unsigned thread, unsigned TX)
{
    return block * (kCausalThreads / TX) + thread / TX;
}

// A worker's way through its share of a channel's rows: pieces in order, row after row.
struct Walk {
    unsigned made, all, left;            // left: pieces that are still its own
    int n, seg, end;
    int64_t t;                          // of the piece's first run, were the row on 16 bytes
    bool on;

    __host__ __device__ __forceinline__ Walk(const CausalArgs &a, unsigned split, int c, bool there) : made(0), t(0)
    {
        const unsigned items = (unsigned)a.N * (unsigned)a.segs;
        all = (items + a.splits - 1) / a.splits;
        const unsigned first = min(items, split * all);
        left = there ? min(items - first, all) : 0;
        on = left > 0;
        n = on ? (int)(first / (unsigned)a.segs) : 0;
        seg = on ? (int)(first - (unsigned)n * a.segs) : 0;
        end = on ? causal_end(a, n) : 0;
    }
    template <typename F>
    __host__ __device__ __forceinline__ void step(const CausalArgs &a, int width, F next_row)
    {
        ++made;
        ++seg;
        t += width;
        on = made < left;
        if (seg == a.segs) {
            seg = 0;
            t = 0;
            ++n;
            next_row();
            end = on ? causal_end(a, n) : 0;
        } else if (!on) {
            end = 0;
        }
    }
};

template <typename T, int K, bool VEC>
__global__ void __launch_bounds__(kCausalThreads) causal_fwd_kernel(const __grid_constant__ CausalArgs a)
{
    constexpr int V = 16 / (int)sizeof(T), M = 2 * V, H = K - 1;
    const unsigned worker = worker_of(blockIdx.x, threadIdx.x, (unsigned)a.TX), tx = threadIdx.x % a.TX;
    const int c = (int)(worker / (unsigned)a.splits);
    const unsigned split = worker % (unsigned)a.splits;
    const bool there = c < a.C;
    ptx::griddep_wait();
    float w[K];
    #pragma unroll
    for (int k = 0; k < K; ++k) w[k] = there ? a.w[(int64_t)c * K + k] : 0.f;
    const float bias = a.bias && there ? a.bias[c] : 0.f;
    Walk at(a, split, c, there);
    at.t = (int64_t)at.seg * a.TX * M;
    const T *row = static_cast<const T *>(a.x) + at.n * a.sx + (int64_t)c * a.L;
    T *out = static_cast<T *>(a.out) + at.n * a.sy + (int64_t)c * a.L;
    // every lane of a warp makes the same rounds: state_out needs the warp together
    for (; at.made < at.all; at.step(a, a.TX * M, [&] { row += a.sx; out += a.sy; })) {
        const bool on = at.on;
        const int n = at.n, end = at.end, phase = VEC ? phase_of(row) : 0;
        const T *state = a.state && H && on ? static_cast<const T *>(a.state) + ((int64_t)n * a.C + c) * H : nullptr;
        const int64_t t_ = at.t + (int64_t)tx * M - phase;
        const int t = on && t_ < a.L ? (int)t_ : a.L;
        const bool whole = VEC && whole_run<T, M, H>(t, end, a.L, state != nullptr);
        if (VEC && on) {                            // the next round's lines, on their way to L2
            if (t_ + a.TX * M < a.L) fetch(row + t_ + a.TX * M);
            else if (at.seg + 1 == a.segs && n + 1 < a.N && (int64_t)tx * M < a.L) fetch(row + a.sx + tx * M);
        }
        if (t < a.L) {
            float win[H + M], y[M];
            load_window<T, M, H, VEC>(row, state, t, end, whole, first_place<T>(phase), win, nullptr, y);
            #pragma unroll
            for (int j = 0; j < M; ++j) {
                float v = bias;
                #pragma unroll
                for (int k = 0; k < K; ++k) v = fmaf(w[k], win[j + k], v);
                y[j] = v;
            }
            if (a.act == GCONV_ACT_SILU) {
                #pragma unroll
                for (int j = 0; j < M; ++j) y[j] *= scan_sigmoid(y[j]);
            }
            if (t + M > end) {
                #pragma unroll
                for (int j = 0; j < M; ++j) y[j] = t + j < end ? y[j] : 0.f;
            }
            store_pieces<T, M, VEC>(out, t, a.L, whole, y);
        }
        if (H && a.state_out) {
            // only a row's first piece reads the state, and its lanes are through with that before the first of them
            // writes: it may be the same memory
            const bool writes = on && at.seg == 0 && tx == 0;
            float last[H ? H : 1];
            #pragma unroll
            for (int j = 0; j < H; ++j) {
                const int at = end - H + j;
                last[j] = !writes ? 0.f : at >= 0 ? to_f(row[at]) : state ? to_f(state[H + at]) : 0.f;
            }
            __syncwarp();
            #pragma unroll
            for (int j = 0; j < H; ++j)
                if (writes) static_cast<T *>(a.state_out)[((int64_t)n * a.C + c) * H + j] = from_f<T>(last[j]);
        }
    }
}

// A few positions (a new one of every sequence): a thread a row, its window in registers.
template <typename T, int K>
__global__ void __launch_bounds__(128) causal_short_kernel(const __grid_constant__ CausalArgs a)
{
    constexpr int H = K - 1;
    const unsigned r_ = blockIdx.x * 128u + threadIdx.x;
    if (r_ >= (unsigned)a.N * (unsigned)a.C) return;
    const int64_t r = r_;
    const int n = (int)(r_ / (unsigned)a.C), c = (int)(r_ % (unsigned)a.C);
    ptx::griddep_wait();
    const int end = causal_end(a, n);
    const T *row = static_cast<const T *>(a.x) + n * a.sx + (int64_t)c * a.L;
    T *out = static_cast<T *>(a.out) + n * a.sy + (int64_t)c * a.L;
    float w[K], win[K];
    #pragma unroll
    for (int k = 0; k < K; ++k) w[k] = a.w[(int64_t)c * K + k];
    const float bias = a.bias ? a.bias[c] : 0.f;
    #pragma unroll
    for (int j = 0; j < H; ++j) win[j] = a.state ? to_f(static_cast<const T *>(a.state)[r * H + j]) : 0.f;
    #pragma unroll
    for (int t = 0; t < kCausalShort; ++t) {
        if (t >= a.L) break;
        float v = 0.f;
        if (t < end) {
            win[H] = to_f(row[t]);
            v = bias;
            #pragma unroll
            for (int k = 0; k < K; ++k) v = fmaf(w[k], win[k], v);
            if (a.act == GCONV_ACT_SILU) v *= scan_sigmoid(v);
            #pragma unroll
            for (int j = 0; j < H; ++j) win[j] = win[j + 1];
        }
        out[t] = from_f<T>(v);
    }
    if (a.state_out) {
        #pragma unroll
        for (int j = 0; j < H; ++j) static_cast<T *>(a.state_out)[r * H + j] = from_f<T>(win[j]);
    }
}

// The last K - 1 positions of dx in a worker's pieces, of a channel with a weight that is infinite or NaN.  The gradient's kernel sums
// over all taps, with zeros for dv behind the end; what is not there has to take no part whatever its weight is.  Told apart in
// that kernel's loop instead it took 71.4 us for 70.1 and, in fp32, 78.3 for 75.4 ([8,2048,2048], 4 taps).
template <typename T>
__device__ __noinline__ void causal_ends_again(const CausalArgs &a, int K, int c, unsigned split, int tx, int width, bool vec)
{
    const int H = K - 1;
    const float *w = a.w + (int64_t)c * K;
    Walk at(a, split, c, true);
    at.t = (int64_t)at.seg * width;
    for (; at.on; at.step(a, width, [] {})) {
        const T *row = static_cast<const T *>(a.x) + at.n * a.sx + (int64_t)c * a.L;
        const T *grad = static_cast<const T *>(a.dy) + at.n * a.sdy + (int64_t)c * a.L;
        const T *state = a.state ? static_cast<const T *>(a.state) + ((int64_t)at.n * a.C + c) * H : nullptr;
        const T *more = a.dstate_out ? static_cast<const T *>(a.dstate_out) + ((int64_t)at.n * a.C + c) * H : nullptr;
        const int64_t begin = at.t - (vec ? phase_of(row) : 0);
        const int from = (int)max((int64_t)max(at.end - H, 0), begin), to = (int)min((int64_t)at.end, begin + width);
        for (int p = from + tx; p < to; p += a.TX) {
            float sum = 0.f;
            for (int k = 0; k < K; ++k) {
                const int r = p + H - k;            // dx[p] += w[k] dv[r]
                if (r >= at.end) continue;
                float dv = to_f(grad[r]);
                if (a.act == GCONV_ACT_SILU) {
                    float v = a.bias ? a.bias[c] : 0.f;
                    for (int j = 0; j < K; ++j) {
                        const int q = r - H + j;
                        v = fmaf(w[j], q >= 0 ? to_f(row[q]) : state ? to_f(state[H + q]) : 0.f, v);
                    }
                    const float s = scan_sigmoid(v);
                    dv *= s * fmaf(v, 1.f - s, 1.f);
                }
                sum = fmaf(w[k], dv, sum);
            }
            if (more && p >= at.end - H) sum += to_f(more[p - (at.end - H)]);
            static_cast<T *>(a.out)[at.n * a.sdx + (int64_t)c * a.L + p] = from_f<T>(sum);
        }
    }
}

// Gradients.  dv of the next lane's first positions comes by shuffles.  Where a row has more pieces than one, a worker's last
// lane makes its dv for the lane before alone, and its run is the first of the next piece: 31 of 32 lanes' work counts.
// (Exchanging through shared memory by the whole block instead took a barrier a piece: 132 us against 99 then.)  Now 70 us for
// [8,2048,2048] bf16, 4 taps: issue slots 0.68, 2.9 TB/s.  Six blocks an SM leave 80 registers: from 5 taps on rows that take 16-byte
// accesses spill (24 to 128 bytes stored).
template <typename T, int K, bool VEC>
__global__ void __launch_bounds__(kCausalThreads, 6) causal_bwd_kernel(const __grid_constant__ CausalArgs a)
{
    constexpr int M = kCausalBack, H = K - 1;
    static_assert(H <= M, "what a lane needs from the next one is in that one's run");
    const unsigned worker = worker_of(blockIdx.x, threadIdx.x, (unsigned)a.TX), tx = threadIdx.x % a.TX;
    const int c = (int)(worker / (unsigned)a.splits), runs = a.segs > 1 ? a.TX - 1 : a.TX;
    const unsigned split = worker % (unsigned)a.splits;
    const bool there = c < a.C;
    ptx::griddep_wait();
    float w[K], dw[K], db = 0.f;
    #pragma unroll
    for (int k = 0; k < K; ++k) { w[k] = there ? a.w[(int64_t)c * K + k] : 0.f; dw[k] = 0.f; }
    const float bias = a.bias && there ? a.bias[c] : 0.f;
    Walk at(a, split, c, there);
    at.t = (int64_t)at.seg * runs * M;
    const T *row = static_cast<const T *>(a.x) + at.n * a.sx + (int64_t)c * a.L;
    const T *grad = static_cast<const T *>(a.dy) + at.n * a.sdy + (int64_t)c * a.L;
    T *out = static_cast<T *>(a.out) + at.n * a.sdx + (int64_t)c * a.L;
    const bool mine = (int)tx < runs;
    // every lane of a warp makes the same rounds, for the shuffles
    for (; at.made < at.all; at.step(a, runs * M, [&] { row += a.sx; grad += a.sdy; out += a.sdx; })) {
        const bool on = at.on;
        const int n = at.n, end = at.end, phase = VEC ? phase_of(row) : 0;
        const T *state = a.state && H && on ? static_cast<const T *>(a.state) + ((int64_t)n * a.C + c) * H : nullptr;
        const int64_t t_ = at.t + (int64_t)tx * M - phase;
        const int t = on && t_ < a.L ? (int)t_ : a.L;
        const T *more = a.dstate_out && on ? static_cast<const T *>(a.dstate_out) + ((int64_t)n * a.C + c) * H : nullptr;
        const bool whole = VEC && (!more || t + M <= end - H) && whole_run<T, M, H>(t, end, a.L, state != nullptr);
        if (VEC && on) {                            // the next round's lines, on their way to L2
            if (t_ + runs * M < a.L) {
                fetch(row + t_ + runs * M);
                fetch(grad + t_ + runs * M);
            } else if (at.seg + 1 == a.segs && n + 1 < a.N && (int64_t)tx * M < a.L) {
                fetch(row + a.sx + tx * M);
                fetch(grad + a.sdy + tx * M);
            }
        }
        float dv[M + H], win[H + M], d[M];
        if (t < end) {
            load_window<T, M, H, VEC>(row, state, t, end, whole, first_place<T>(phase), win, grad, d);
            if (a.act == GCONV_ACT_SILU) {
                #pragma unroll
                for (int j = 0; j < M; ++j) {
                    float v = bias;
                    #pragma unroll
                    for (int k = 0; k < K; ++k) v = fmaf(w[k], win[j + k], v);
                    const float s = scan_sigmoid(v);
                    dv[j] = d[j] * (s * fmaf(v, 1.f - s, 1.f));
                }
            } else {
                #pragma unroll
                for (int j = 0; j < M; ++j) dv[j] = d[j];
            }
            if (whole) {
                if (mine) {
                    #pragma unroll
                    for (int j = 0; j < M; ++j) {
                        db += dv[j];
                        #pragma unroll
                        for (int k = 0; k < K; ++k) dw[k] = fmaf(dv[j], win[j + k], dw[k]);
                    }
                }
            } else {
                #pragma unroll
                for (int j = 0; j < M; ++j) {
                    const bool in = t + j >= 0 && t + j < end;
                    dv[j] = in ? dv[j] : 0.f;
                    if (!in || !mine) continue;
                    db += dv[j];
                    #pragma unroll
                    for (int k = 0; k < K; ++k) dw[k] = fmaf(dv[j], win[j + k], dw[k]);
                }
            }
        } else {
            #pragma unroll
            for (int j = 0; j < M; ++j) dv[j] = 0.f;
        }
        #pragma unroll
        for (int j = 0; j < H; ++j) {
            const float next = __shfl_down_sync(~0u, dv[j], 1);
            dv[M + j] = (int)tx + 1 < a.TX ? next : 0.f;
        }
        if (on && mine && t < a.L) {
            float dx[M];
            #pragma unroll
            for (int j = 0; j < M; ++j) {
                float v = 0.f;
                #pragma unroll
                for (int k = 0; k < K; ++k) v = fmaf(w[k], dv[j + H - k], v);
                dx[j] = v;
            }
            if (t + M > end - H) {                   // near the end, or behind it
                #pragma unroll
                for (int j = 0; j < M; ++j) {
                    const int from = t + j - (end - H);
                    if (H && more && from >= 0 && from < H) dx[j] += to_f(more[from]);
                    dx[j] = t + j < end ? dx[j] : 0.f;
                }
            }
            store_pieces<T, M, VEC>(out, t, a.L, whole, dx);
            if (H && a.dstate && at.seg == 0 && tx == 0) {
                #pragma unroll
                for (int j = 0; j < H; ++j) {
                    float v = 0.f;
                    #pragma unroll
                    for (int k = 0; k <= j; ++k) {
                        #pragma unroll
                        for (int m = 0; m < M + H; ++m)
                            if (t + m == j - k && j - k < end) v = fmaf(w[k], dv[m], v);
                    }
                    if (more && j - end >= 0 && j - end < H) v += to_f(more[j - end]);
                    static_cast<T *>(a.dstate)[((int64_t)n * a.C + c) * H + j] = from_f<T>(v);
                }
            }
        }
    }
    #pragma unroll
    for (int k = 0; k <= K; ++k) {
        float v = k < K ? dw[k < K ? k : 0] : db;
        for (int o = a.TX / 2; o > 0; o >>= 1) v += __shfl_down_sync(~0u, v, o, a.TX);
        if (tx == 0 && there) a.part[((int64_t)split * a.C + c) * (K + 1) + k] = v;
    }
    float odd = 0.f;
    #pragma unroll
    for (int k = 0; k < K; ++k) odd = fmaf(w[k], 0.f, odd);
    __syncwarp();                                   // a row's end may be another lane's
    if (H && odd != 0.f) causal_ends_again<T>(a, K, c, split, (int)tx, runs * M, VEC);
}

// dw and db from the workers' sums, in order: 32 columns a block, eight threads a column.
__global__ void __launch_bounds__(256) causal_sum_kernel(const float *part, int splits, int C, int K, float *dw, float *db)
{
    __shared__ float sh[8][32];
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t cols = (int64_t)C * (K + 1), col = (int64_t)blockIdx.x * 32 + lane;
    float v = 0.f;
    if (col < cols)
        for (int s = k; s < splits; s += 8) v += part[s * cols + col];
    sh[k][lane] = v;
    __syncthreads();
    if (k || col >= cols) return;
    #pragma unroll
    for (int j = 1; j < 8; ++j) v += sh[j][lane];
    const int c = (int)(col / (K + 1)), at = (int)(col % (K + 1));
    if (at < K) dw[(int64_t)c * K + at] = v;
    else if (db) db[c] = v;
}

// ---- checks and launches ----------------------------------------------------------------

int esize(gconv_dtype dt) { return dt == GCONV_BF16 ? 2 : 4; }
bool on(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool check_causal(const gconv_causal *s, gconv_dtype dt)
{
    if (!s || (dt != GCONV_F32 && dt != GCONV_BF16)) return false;
    if (s->N < 0 || s->C < 1 || s->L < 1 || s->L > (1 << 30) || s->taps < 1 || s->taps > kCausalMost) return false;
    if (s->act != GCONV_ACT_NONE && s->act != GCONV_ACT_SILU) return false;
    const int64_t CL = (int64_t)s->C * s->L;
    if (CL > ((int64_t)1 << 40) / std::max(1, s->N) || (int64_t)s->N * s->C > INT_MAX) return false;
    for (long long b : {s->x_batch, s->y_batch, s->dy_batch, s->dx_batch})
        if (b != 0 && (b < CL || b > ((int64_t)1 << 40))) return false;
    return true;
}

struct CausalShape { int TX, segs, splits; int64_t grid; };

// `whole`: every row begins on 16 bytes.
CausalShape causal_shape(const gconv_causal &s, gconv_dtype dt, bool back, bool whole)
{
    const int V = 16 / esize(dt), M = back ? kCausalBack : 2 * V;
    // lanes of a worker and pieces of a row of `n` runs: as few lanes idle as may be, then the most lanes
    auto cut = [&](int64_t n, int64_t *segs) {
        int best = 1;
        int64_t least = 0;
        for (int TX = 32; TX >= 1; TX /= 2) {
            const int64_t each = back && n > TX ? TX - 1 : TX;
            if (each < 1 || (n > TX && TX < 8)) continue;
            const int64_t pieces = (n + each - 1) / each;
            if (least == 0 || pieces * TX < least) { least = pieces * TX; best = TX; *segs = pieces; }
        }
        return best;
    };
    int64_t segs = 1, usual = 1;
    CausalShape p{};
    p.TX = cut(((int64_t)s.L + (whole ? 0 : V - 1) + M - 1) / M, &segs);
    p.segs = (int)segs;
    // workers that share a channel: 64 warps an SM; the workspace's size does not know the alignment, so they go by rows that begin
    // anywhere.  Forward and gradient in us with 32, 64 and 128, 4 taps: [8,2048,2048] bf16 30 and 71, 32 and 70, 37 and 77;
    // [1,2048,4096] bf16 10 and 20, 14 and 22, 20 and 26; [64,2048,64] bf16 9.7 and 24, 9.0 and 24, 9.4 and 25; [7,512,1023] fp32 8.3
    // and 17.5, 8.2 and 17.5, 8.1 and 19
    const int lanes = cut(((int64_t)s.L + V - 1 + M - 1) / M, &usual);
    const int64_t want = (int64_t)num_sms() * 64 * (32 / lanes);
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>((int64_t)s.N * usual, (want + s.C - 1) / s.C));
    p.grid = ((int64_t)s.C * p.splits + kCausalThreads / p.TX - 1) / (kCausalThreads / p.TX);
    return p;
}

void causal_args(const gconv_causal &s, CausalArgs *a)
{
    const int64_t CL = (int64_t)s.C * s.L;
    a->N = s.N; a->C = s.C; a->L = s.L; a->act = s.act;
    a->sx = s.x_batch ? s.x_batch : CL; a->sy = s.y_batch ? s.y_batch : CL;
    a->sdy = s.dy_batch ? s.dy_batch : CL; a->sdx = s.dx_batch ? s.dx_batch : CL;
}

// Whether rows of both tensors always begin at the same place of a 16-byte piece.
bool together(const gconv_causal &s, gconv_dtype dt, const void *p, int64_t sp, const void *q, int64_t sq)
{
    const int E = 16 / esize(dt);
    return ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0 && (s.N == 1 || (sp - sq) % E == 0);
}

bool whole_rows(const gconv_causal &s, gconv_dtype dt, const void *p, int64_t sp)
{
    const int E = 16 / esize(dt);
    return on(p, 16) && s.L % E == 0 && (s.N == 1 || sp % E == 0);
}

template <typename T, int K = 1>
void causal_start(int K_, int kind, bool vec, const CausalArgs &a, int64_t grid, cudaStream_t st)
{
    if (K_ == K) {
        if (kind == 0) launch_dependent(causal_short_kernel<T, K>, (unsigned)grid, 128u, 0, st, a);
        else if (kind == 1 && vec) launch_dependent(causal_fwd_kernel<T, K, true>, (unsigned)grid, (unsigned)kCausalThreads, 0, st, a);
        else if (kind == 1) launch_dependent(causal_fwd_kernel<T, K, false>, (unsigned)grid, (unsigned)kCausalThreads, 0, st, a);
        else if (vec) launch_dependent(causal_bwd_kernel<T, K, true>, (unsigned)grid, (unsigned)kCausalThreads, 0, st, a);
        else launch_dependent(causal_bwd_kernel<T, K, false>, (unsigned)grid, (unsigned)kCausalThreads, 0, st, a);
        return;
    }
    if constexpr (K < kCausalMost) causal_start<T, K + 1>(K_, kind, vec, a, grid, st);
}

size_t causal_ws(const gconv_causal &s, gconv_dtype dt)
{
    return s.N ? (size_t)causal_shape(s, dt, true, false).splits * s.C * (s.taps + 1) * sizeof(float) : 0;
}

gconv_status done() { return cudaGetLastError() == cudaSuccess ? GCONV_OK : GCONV_ERR_CUDA; }

}  // namespace

}  // namespace gconv

using namespace gconv;

extern "C" {

size_t gconv_causal_workspace_size(const gconv_causal *causal, gconv_dtype dtype)
{
    return check_causal(causal, dtype) ? causal_ws(*causal, dtype) : (size_t)-1;
}

gconv_status gconv_causal_fwd(const gconv_causal *causal, gconv_dtype dtype, const void *x, const float *w, const float *bias,
                              const void *state, const int *lengths, void *y, void *state_out, void *stream)
{
    if (!check_causal(causal, dtype)) return GCONV_ERR_INVALID_ARG;
    if (causal->N == 0) return GCONV_OK;
    const int es = esize(dtype);
    if (!x || !w || !y || !on(x, es) || !on(y, es) || !on(state, es) || !on(state_out, es)) return GCONV_ERR_INVALID_ARG;
    if (!on(w, 4) || !on(bias, 4) || !on(lengths, 4)) return GCONV_ERR_INVALID_ARG;
    CausalArgs a{};
    causal_args(*causal, &a);
    const bool vec = together(*causal, dtype, x, a.sx, y, a.sy);
    const CausalShape p = causal_shape(*causal, dtype, false, !vec || whole_rows(*causal, dtype, x, a.sx));
    a.TX = p.TX; a.segs = p.segs; a.splits = p.splits;
    a.x = x; a.w = w; a.bias = bias; a.state = state; a.state_out = causal->taps > 1 ? state_out : nullptr; a.lengths = lengths;
    a.out = y;
    const bool brief = causal->L <= kCausalShort;
    const int64_t grid = brief ? ((int64_t)a.N * a.C + 127) / 128 : p.grid;
    if (grid > INT_MAX || (int64_t)causal->N * p.segs > INT_MAX) return GCONV_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == GCONV_BF16) causal_start<__nv_bfloat16>(causal->taps, brief ? 0 : 1, vec, a, grid, st);
    else causal_start<float>(causal->taps, brief ? 0 : 1, vec, a, grid, st);
    return done();
}

gconv_status gconv_causal_bwd(const gconv_causal *causal, gconv_dtype dtype, const void *x, const float *w, const float *bias,
                              const void *state, const int *lengths, const void *dy, const void *dstate_out, void *dx,
                              float *dw, float *dbias, void *dstate, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!check_causal(causal, dtype) || !w || !dw || !on(w, 4) || !on(bias, 4) || !on(lengths, 4) || !on(dw, 4) || !on(dbias, 4))
        return GCONV_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (causal->N == 0) {
        const size_t c = (size_t)causal->C * sizeof(float);
        if (cudaMemsetAsync(dw, 0, c * causal->taps, st) != cudaSuccess || (dbias && cudaMemsetAsync(dbias, 0, c, st) != cudaSuccess))
            return GCONV_ERR_CUDA;
        return GCONV_OK;
    }
    const int es = esize(dtype);
    if (!x || !dy || !dx) return GCONV_ERR_INVALID_ARG;
    for (const void *q : {x, dy, state, dstate_out, (const void *)dx, (const void *)dstate})
        if (!on(q, es)) return GCONV_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < causal_ws(*causal, dtype) || !on(workspace, 16)) return GCONV_ERR_WORKSPACE;
    CausalArgs a{};
    causal_args(*causal, &a);
    const bool vec = together(*causal, dtype, x, a.sx, dy, a.sdy) && together(*causal, dtype, x, a.sx, dx, a.sdx);
    const CausalShape p = causal_shape(*causal, dtype, true, !vec || whole_rows(*causal, dtype, x, a.sx));
    if (p.grid > INT_MAX || (int64_t)causal->N * p.segs > INT_MAX) return GCONV_ERR_INVALID_ARG;
    a.TX = p.TX; a.segs = p.segs; a.splits = p.splits;
    const bool held = causal->taps > 1;
    a.x = x; a.w = w; a.bias = bias; a.state = state; a.lengths = lengths; a.dy = dy; a.out = dx;
    a.dstate_out = held ? dstate_out : nullptr; a.dstate = held ? dstate : nullptr;
    a.part = static_cast<float *>(workspace);
    if (dtype == GCONV_BF16) causal_start<__nv_bfloat16>(causal->taps, 2, vec, a, p.grid, st);
    else causal_start<float>(causal->taps, 2, vec, a, p.grid, st);
    const int64_t cols = (int64_t)a.C * (causal->taps + 1);
    launch_dependent(causal_sum_kernel, (unsigned)((cols + 31) / 32), 256u, 0, st, static_cast<const float *>(a.part), p.splits, a.C,
                     causal->taps, dw, dbias);
    return done();
}

}  // extern "C"
