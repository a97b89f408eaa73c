// causal.cu -- short causal convolution along the positions of each channel, and its gradients.
//
//   v[t] = bias + sum_k w[k] x[t - K + 1 + k],   y = act(v),   x before position 0 from the state
//   dv = dy act'(v),   dx[t] = sum_k w[k] dv[t + K - 1 - k],   dw[k] = sum dv[t] x[t - K + 1 + k],   db = sum dv
//
// Two or three tensors go through once, at 2 K + 8 operations an element, so memory bounds it: every access is 16 bytes.
// A thread takes the elements of one row (channel of a sequence) that lie in one aligned 16-byte piece of memory, so rows of
// odd length, which begin anywhere, are read in whole pieces too; only a row's two ends go element by element.  What
// the window needs from the pieces beside it is read again (from L1).
#include "scan.cuh"

#include <algorithm>
#include <climits>

namespace gconv {

namespace {

constexpr int kCausalMost = 8;          // taps
constexpr int kCausalShort = 4;         // positions of the form with one thread a row
constexpr int kCausalThreads = 256;

struct CausalArgs {
    int N, C, L, act;
    int TX, segs;                       // threads of a row in a block (a power of two), pieces of a row
    int splits;                         // gradient: blocks that share a channel
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

__device__ __forceinline__ int causal_end(const CausalArgs &a, int n)
{
    if (!a.lengths) return a.L;
    const int v = a.lengths[n];
    return v < 0 ? 0 : v < a.L ? v : a.L;
}

// Elements t .. t + V - 1 of a row, zeros outside [0, end); an address on 16 bytes where VEC.
template <typename T, int V, bool VEC>
__device__ __forceinline__ void load_piece(const T *row, int t, int end, float (&v)[V])
{
    if (VEC && t >= 0 && t + V <= end) {
        const Pack<T, V> x = *reinterpret_cast<const Pack<T, V> *>(row + t);
        #pragma unroll
        for (int j = 0; j < V; ++j) v[j] = to_f(x.v[j]);
    } else {
        #pragma unroll
        for (int j = 0; j < V; ++j) v[j] = t + j >= 0 && t + j < end ? to_f(row[t + j]) : 0.f;
    }
}

template <typename T, int V, bool VEC>
__device__ __forceinline__ void store_piece(T *row, int t, int L, const float (&v)[V])
{
    if (VEC && t >= 0 && t + V <= L) {
        Pack<T, V> x;
        #pragma unroll
        for (int j = 0; j < V; ++j) x.v[j] = from_f<T>(v[j]);
        *reinterpret_cast<Pack<T, V> *>(row + t) = x;
    } else {
        #pragma unroll
        for (int j = 0; j < V; ++j)
            if (t + j >= 0 && t + j < L) row[t + j] = from_f<T>(v[j]);
    }
}

// win[i]: x at t - H + i for i < H + V (zeros outside the sequence, the state before it).
template <typename T, int V, int H, bool VEC>
__device__ __forceinline__ void load_window(const T *row, const T *state, int t, int end, float (&win)[H + V])
{
    float cur[V];
    load_piece<T, V, VEC>(row, t, end, cur);
    #pragma unroll
    for (int j = 0; j < V; ++j) win[H + j] = cur[j];
    #pragma unroll
    for (int b = 1; b <= (H + V - 1) / V; ++b) {
        float old[V];
        load_piece<T, V, VEC>(row, t - b * V, end, old);
        #pragma unroll
        for (int j = 0; j < V; ++j)
            if (H - b * V + j >= 0) win[H - b * V + j] = old[j];
    }
    if (state) {
        #pragma unroll
        for (int i = 0; i < H + V; ++i) {
            const int at = t - H + i;
            if (at < 0 && at >= -H) win[i] = to_f(state[H + at]);
        }
    }
}

template <typename T>
__device__ __forceinline__ int phase_of(const T *row)
{
    return (int)((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % (16 / sizeof(T)));
}

template <typename T, int K, bool VEC>
__global__ void __launch_bounds__(kCausalThreads) causal_fwd_kernel(const CausalArgs a)
{
    constexpr int V = 16 / (int)sizeof(T), H = K - 1;
    const int seg = (int)(blockIdx.x % a.segs);
    const int64_t r = (int64_t)(blockIdx.x / a.segs) * (kCausalThreads / a.TX) + threadIdx.x / a.TX;
    const bool there = r < (int64_t)a.N * a.C;
    const int n = there ? (int)(r / a.C) : 0, c = there ? (int)(r % a.C) : 0;
    const int i = seg * a.TX + threadIdx.x % a.TX;
    ptx::griddep_wait();
    const int end = there ? causal_end(a, n) : 0;
    const T *row = static_cast<const T *>(a.x) + n * a.sx + (int64_t)c * a.L;
    T *out = static_cast<T *>(a.out) + n * a.sy + (int64_t)c * a.L;
    const T *state = a.state && H ? static_cast<const T *>(a.state) + ((int64_t)n * a.C + c) * H : nullptr;
    const int t = i * V - (VEC ? phase_of(row) : 0);
    float win[H + V];
    if (there && t < a.L) {
        load_window<T, V, H, VEC>(row, state, t, end, win);
        float w[K], y[V];
        #pragma unroll
        for (int k = 0; k < K; ++k) w[k] = a.w[(int64_t)c * K + k];
        const float bias = a.bias ? a.bias[c] : 0.f;
        #pragma unroll
        for (int j = 0; j < V; ++j) {
            float v = bias;
            #pragma unroll
            for (int k = 0; k < K; ++k) v = fmaf(w[k], win[j + k], v);
            if (a.act == GCONV_ACT_SILU) v *= scan_sigmoid(v);
            y[j] = t + j < end ? v : 0.f;
        }
        store_piece<T, V, VEC>(out, t, a.L, y);
    }
    if (H && a.state_out && seg == 0) {
        // the window's reads of the state are over before any thread of the row writes it: it may be the same memory
        float last[H ? H : 1];
        const bool writes = there && i == 0;
        #pragma unroll
        for (int j = 0; j < H; ++j) {
            const int at = end - H + j;
            last[j] = !writes ? 0.f : at >= 0 ? to_f(row[at]) : state ? to_f(state[H + at]) : 0.f;
        }
        __syncthreads();
        #pragma unroll
        for (int j = 0; j < H; ++j)
            if (writes) static_cast<T *>(a.state_out)[r * H + j] = from_f<T>(last[j]);
    }
}

// A few positions (a new one of every sequence): a thread a row, its window in registers.
template <typename T, int K>
__global__ void __launch_bounds__(128) causal_short_kernel(const CausalArgs a)
{
    constexpr int H = K - 1;
    const int64_t r = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (r >= (int64_t)a.N * a.C) return;
    const int n = (int)(r / a.C), c = (int)(r % a.C);
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

// Gradients.  A block takes TY channels and walks over its share of the sequences and row pieces; dw and db stay in
// registers until the end.  dv of the next thread's first positions comes through shared memory; the last thread of a
// row's piece makes it itself.
template <typename T, int K, bool VEC>
__global__ void __launch_bounds__(kCausalThreads) causal_bwd_kernel(const CausalArgs a)
{
    constexpr int V = 16 / (int)sizeof(T), H = K - 1;
    __shared__ float ahead[2][H ? H : 1][kCausalThreads];
    __shared__ float sums[kCausalThreads / 32][K + 1];
    const int TY = kCausalThreads / a.TX, tx = threadIdx.x % a.TX;
    const int c = (int)(blockIdx.x / a.splits) * TY + threadIdx.x / a.TX, split = (int)(blockIdx.x % a.splits);
    const bool there = c < a.C;
    ptx::griddep_wait();
    float w[K], dw[K], db = 0.f;
    #pragma unroll
    for (int k = 0; k < K; ++k) { w[k] = there ? a.w[(int64_t)c * K + k] : 0.f; dw[k] = 0.f; }
    const float bias = a.bias && there ? a.bias[c] : 0.f;
    int turn = 0;
    const int64_t items = (int64_t)a.N * a.segs;
    for (int64_t item = split; item < items; item += a.splits, turn ^= 1) {
        const int n = (int)(item / a.segs), seg = (int)(item % a.segs);
        const int i = seg * a.TX + tx, end = there ? causal_end(a, n) : 0;
        const T *row = static_cast<const T *>(a.x) + n * a.sx + (int64_t)c * a.L;
        const T *grad = static_cast<const T *>(a.dy) + n * a.sdy + (int64_t)c * a.L;
        const T *state = a.state && H && there ? static_cast<const T *>(a.state) + ((int64_t)n * a.C + c) * H : nullptr;
        const int t = i * V - (VEC && there ? phase_of(row) : 0);
        const bool any = t < end;
        float dv[V + H], win[H + V];
        #pragma unroll
        for (int j = 0; j < V + H; ++j) dv[j] = 0.f;
        auto back = [&](float v, float d) {          // dy act'(v)
            if (a.act != GCONV_ACT_SILU) return d;
            const float s = scan_sigmoid(v);
            return d * (s * fmaf(v, 1.f - s, 1.f));
        };
        if (any) {
            float d[V];
            load_window<T, V, H, VEC>(row, state, t, end, win);
            load_piece<T, V, VEC>(grad, t, end, d);
            #pragma unroll
            for (int j = 0; j < V; ++j) {
                float v = bias;
                #pragma unroll
                for (int k = 0; k < K; ++k) v = fmaf(w[k], win[j + k], v);
                const float x = back(v, d[j]);
                dv[j] = t + j >= 0 && t + j < end ? x : 0.f;
                db += dv[j];
                #pragma unroll
                for (int k = 0; k < K; ++k) dw[k] = fmaf(dv[j], win[j + k], dw[k]);
            }
        }
        if constexpr (H > 0) {
            #pragma unroll
            for (int j = 0; j < H; ++j) ahead[turn][j][threadIdx.x] = j < V ? dv[j < V ? j : 0] : 0.f;
            if (V >= H) __syncthreads();
            if (any && (tx == a.TX - 1 || V < H)) {
                #pragma unroll
                for (int j = 0; j < H; ++j) {
                    const int at = t + V + j;
                    if (at >= end) continue;
                    float v = bias;
                    #pragma unroll
                    for (int k = 0; k < K; ++k) {
                        const int from = at - H + k;
                        const float x = from >= 0 ? to_f(row[from]) : state && from >= -H ? to_f(state[H + from]) : 0.f;
                        v = fmaf(w[k], x, v);
                    }
                    if (at >= 0) dv[V + j] = back(v, to_f(grad[at]));
                }
            } else if (any) {
                #pragma unroll
                for (int j = 0; j < H; ++j) dv[V + j] = ahead[turn][j][threadIdx.x + 1];
            }
        }
        if (there && t < a.L) {
            float dx[V];
            const T *more = a.dstate_out ? static_cast<const T *>(a.dstate_out) + ((int64_t)n * a.C + c) * H : nullptr;
            #pragma unroll
            for (int j = 0; j < V; ++j) {
                float v = 0.f;
                #pragma unroll
                for (int k = 0; k < K; ++k) v = fmaf(w[k], dv[j + H - k], v);
                const int from = t + j - (end - H);
                if (H && more && from >= 0 && from < H) v += to_f(more[from]);
                dx[j] = t + j < end ? v : 0.f;
            }
            store_piece<T, V, VEC>(static_cast<T *>(a.out) + n * a.sdx + (int64_t)c * a.L, t, a.L, dx);
            if (H && a.dstate && i == 0) {
                #pragma unroll
                for (int j = 0; j < H; ++j) {
                    float v = 0.f;
                    #pragma unroll
                    for (int k = 0; k <= j; ++k) {
                        #pragma unroll
                        for (int m = 0; m < V + H; ++m)
                            if (t + m == j - k) v = fmaf(w[k], dv[m], v);
                    }
                    if (more && j - end >= 0 && j - end < H) v += to_f(more[j - end]);
                    static_cast<T *>(a.dstate)[((int64_t)n * a.C + c) * H + j] = from_f<T>(v);
                }
            }
        }
    }
    // over the TX threads of a channel: a warp's by shuffles, the warps' in order
    const int width = a.TX < 32 ? a.TX : 32;
    #pragma unroll
    for (int k = 0; k <= K; ++k) {
        float v = k < K ? dw[k < K ? k : 0] : db;
        for (int o = width / 2; o > 0; o >>= 1) v += __shfl_down_sync(~0u, v, o, width);
        if (a.TX <= 32) {
            if (tx == 0 && there) a.part[((int64_t)split * a.C + c) * (K + 1) + k] = v;
        } else if ((threadIdx.x & 31) == 0) {
            sums[threadIdx.x >> 5][k] = v;
        }
    }
    if (a.TX > 32) {
        __syncthreads();
        if (there && tx <= K) {
            float v = 0.f;
            for (int j = 0; j < a.TX / 32; ++j) v += sums[threadIdx.x / a.TX * (a.TX / 32) + j][tx];
            a.part[((int64_t)split * a.C + c) * (K + 1) + tx] = v;
        }
    }
}

// dw and db from the blocks' sums, in order: 32 columns a block, eight threads a column.
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
    if (s->N < 0 || s->C < 1 || s->L < 1 || s->taps < 1 || s->taps > kCausalMost) return false;
    if (s->act != GCONV_ACT_NONE && s->act != GCONV_ACT_SILU) return false;
    const int64_t CL = (int64_t)s->C * s->L;
    if (CL > ((int64_t)1 << 40) / std::max(1, s->N)) return false;
    for (long long b : {s->x_batch, s->y_batch, s->dy_batch, s->dx_batch})
        if (b != 0 && (b < CL || b > ((int64_t)1 << 40))) return false;
    return true;
}

struct CausalShape { int TX, segs, splits; int64_t grid; };

CausalShape causal_shape(const gconv_causal &s, gconv_dtype dt, bool back)
{
    const int V = 16 / esize(dt);
    CausalShape p{};
    const int64_t pieces = ((int64_t)s.L + 2 * V - 2) / V;       // of a row that begins anywhere
    p.TX = 1;
    while (p.TX < kCausalThreads && p.TX < pieces) p.TX *= 2;
    p.segs = (int)((pieces + p.TX - 1) / p.TX);
    const int TY = kCausalThreads / p.TX;
    if (!back) {
        p.grid = ((int64_t)s.N * s.C + TY - 1) / TY * p.segs;
        return p;
    }
    const int64_t blocks = (s.C + TY - 1) / TY, items = (int64_t)s.N * p.segs;
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(items, ((int64_t)num_sms() * 16 + blocks - 1) / blocks));
    p.grid = blocks * p.splits;
    return p;
}

void causal_args(const gconv_causal &s, const CausalShape &p, CausalArgs *a)
{
    const int64_t CL = (int64_t)s.C * s.L;
    a->N = s.N; a->C = s.C; a->L = s.L; a->act = s.act;
    a->TX = p.TX; a->segs = p.segs; a->splits = p.splits;
    a->sx = s.x_batch ? s.x_batch : CL; a->sy = s.y_batch ? s.y_batch : CL;
    a->sdy = s.dy_batch ? s.dy_batch : CL; a->sdx = s.dx_batch ? s.dx_batch : CL;
}

// Whether rows of both tensors always begin at the same place of a 16-byte piece.
bool together(const gconv_causal &s, gconv_dtype dt, const void *p, int64_t sp, const void *q, int64_t sq)
{
    const int E = 16 / esize(dt);
    return ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0 && (s.N == 1 || (sp - sq) % E == 0);
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
    return s.N ? (size_t)causal_shape(s, dt, true).splits * s.C * (s.taps + 1) * sizeof(float) : 0;
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
    const CausalShape p = causal_shape(*causal, dtype, false);
    CausalArgs a{};
    causal_args(*causal, p, &a);
    a.x = x; a.w = w; a.bias = bias; a.state = state; a.state_out = causal->taps > 1 ? state_out : nullptr; a.lengths = lengths;
    a.out = y;
    const bool brief = causal->L <= kCausalShort;
    const int64_t grid = brief ? ((int64_t)a.N * a.C + 127) / 128 : p.grid;
    if (grid > INT_MAX) return GCONV_ERR_INVALID_ARG;
    const bool vec = together(*causal, dtype, x, a.sx, y, a.sy);
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
    const CausalShape p = causal_shape(*causal, dtype, true);
    if (p.grid > INT_MAX) return GCONV_ERR_INVALID_ARG;
    CausalArgs a{};
    causal_args(*causal, p, &a);
    const bool held = causal->taps > 1;
    a.x = x; a.w = w; a.bias = bias; a.state = state; a.lengths = lengths; a.dy = dy; a.out = dx;
    a.dstate_out = held ? dstate_out : nullptr; a.dstate = held ? dstate : nullptr;
    a.part = static_cast<float *>(workspace);
    const bool vec = together(*causal, dtype, x, a.sx, dy, a.sdy) && together(*causal, dtype, x, a.sx, dx, a.sdx);
    if (dtype == GCONV_BF16) causal_start<__nv_bfloat16>(causal->taps, 2, vec, a, p.grid, st);
    else causal_start<float>(causal->taps, 2, vec, a, p.grid, st);
    const int64_t cols = (int64_t)a.C * (causal->taps + 1);
    launch_dependent(causal_sum_kernel, (unsigned)((cols + 31) / 32), 256u, 0, st, static_cast<const float *>(a.part), p.splits, a.C,
                     causal->taps, dw, dbias);
    return done();
}

}  // extern "C"
