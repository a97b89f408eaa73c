// newton_tiny.cu -- Newton-Schulz steps of matrices of at most 16 x 1024 (the groups of grouped
// and depthwise layers): one thread block a matrix, fp32 in shared memory from first to last.
//
// A step is three sweeps between block barriers: A (m (m + 1) / 2 dot products of length n, a few
// lanes each), P = a I + b A + c A A, and X <- P X from one copy of X to the other.  With so few
// operations the tensor cores' fill and drain are most of a step's time, and plain fp32 is
// both quicker and exact to fp32.  Bound by the barriers and the shared-memory reads of one block: five
// steps of 32 matrices of 4 x 36 6.7 us, of one or 256 of 8 x 72 8.1 and 8.9.
#include "newton.cuh"

#include <algorithm>

namespace gconv {

namespace {

constexpr int kTinyRows = 16, kTinyCols = 1024, kTinyWork = 32768;

struct TinyParams {
    NewtonIn in;
    NewtonOut out;
    int m, n, ld, steps, lanes, pairs;   // lanes: a power of two a dot product; pairs = m (m + 1) / 2
    float coeffs[3 * kNewtonSteps];
};

__global__ void __launch_bounds__(256) newton_tiny_kernel(const __grid_constant__ TinyParams p)
{
    extern __shared__ __align__(16) float sm[];
    __shared__ __align__(16) float A[kTinyRows][kTinyRows], P[kTinyRows][kTinyRows];
    __shared__ float sums[8];
    __shared__ uint8_t rows_of[kTinyRows * (kTinyRows + 1) / 2][2];
    const int tid = threadIdx.x, threads = blockDim.x, m = p.m, n = p.n, ld = p.ld;
    float *X = sm, *Y = sm + (size_t)kTinyRows * ld;
    const int64_t base = (int64_t)blockIdx.x * p.in.elems;

    if (tid < m)
        for (int j = 0; j <= tid; ++j) {
            rows_of[tid * (tid + 1) / 2 + j][0] = (uint8_t)tid;
            rows_of[tid * (tid + 1) / 2 + j][1] = (uint8_t)j;
        }
    for (int i = tid; i < kTinyRows * kTinyRows; i += threads) A[i / kTinyRows][i % kTinyRows] = P[i / kTinyRows][i % kTinyRows] = 0.f;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    float s = 0.f;
    #pragma unroll 4
    for (int i = tid; i < m * n; i += threads) {
        float u = load_g(p.in, base + i);
        if (p.in.m) {
            const float v = fmaf(p.in.beta, p.in.m[base + i], u);
            p.in.m_out[base + i] = v;
            u = lookahead(p.in, u, v);
        }
        const int r = i / p.in.cols, c = i - r * p.in.cols;
        X[p.in.tall ? c * ld + r : r * ld + c] = u;
        s = fmaf(u, u, s);
    }
    #pragma unroll
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if ((tid & 31) == 0) sums[tid >> 5] = s;
    __syncthreads();
    float total = 0.f;
    for (int k = 0; k < threads / 32; ++k) total += sums[k];
    float inv = unit_factor(1.f, total, p.in.eps);   // of the first X: applied where it is read
    const int lane = tid & (p.lanes - 1), first = tid / p.lanes, hop = threads / p.lanes;
    const int rounds = (p.pairs + hop - 1) / hop, m4 = (m + 3) / 4;

    for (int step = 0; step < p.steps; ++step) {
        const float a = p.coeffs[3 * step], b = p.coeffs[3 * step + 1], c = p.coeffs[3 * step + 2];
        for (int k = 0, q = first; k < rounds; ++k, q += hop) {   // whole warps in every round: the sums shuffle
            float t = 0.f;
            int i = 0, j = 0;
            if (q < p.pairs) {
                i = rows_of[q][0];
                j = rows_of[q][1];
                const float *x = X + i * ld, *y = X + j * ld;
                #pragma unroll 4
                for (int e = lane; e < n; e += p.lanes) t = fmaf(x[e] * inv, y[e] * inv, t);
            }
            for (int o = 1; o < p.lanes; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            if (lane == 0 && q < p.pairs) A[i][j] = A[j][i] = t;
        }
        __syncthreads();
        for (int e = tid; e < m * m; e += threads) {
            const int i = e / m, j = e - i * m;
            float t = 0.f;
            #pragma unroll
            for (int k = 0; k < kTinyRows; ++k) t = fmaf(A[i][k], A[k][j], t);   // zeros past m
            P[i][j] = fmaf(c, t, b * A[i][j]) + (i == j ? a : 0.f);
        }
        __syncthreads();
        for (int e = tid; e < n * m4; e += threads) {
            const int r = e / n, col = e - r * n;
            float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < m; ++k) {
                const float x = X[k * ld + col] * inv;
                const float4 w = *reinterpret_cast<const float4 *>(&P[k][4 * r]);   // P is symmetric
                t.x = fmaf(w.x, x, t.x); t.y = fmaf(w.y, x, t.y); t.z = fmaf(w.z, x, t.z); t.w = fmaf(w.w, x, t.w);
            }
            float *y = Y + 4 * r * ld + col;
            y[0] = t.x; y[ld] = t.y; y[2 * ld] = t.z; y[3 * ld] = t.w;
        }
        __syncthreads();
        inv = 1.f;
        float *swap = X;
        X = Y;
        Y = swap;
    }
    #pragma unroll 4
    for (int i = tid; i < m * n; i += threads) {
        const int r = i / p.in.cols, c = i - r * p.in.cols;
        store_result(p.out, base + i, X[p.in.tall ? c * ld + r : r * ld + c]);
    }
}

}  // namespace

// A step's time grows with m^2 n and the cluster kernel's hardly does.  Measured, one matrix, here
// against there: 8 x 72 8 us and 18, 16 x 256 30 and 19, 16 x 1024 105 and 21.
bool newton_tiny_fits(const NewtonShape &s)
{
    return s.m <= kTinyRows && s.n <= kTinyCols && s.m * s.m * s.n <= kTinyWork;
}

gconv_status newton_tiny_launch(const NewtonShape &s, const NewtonIn &in, const NewtonOut &out, int steps,
                                const float *coeffs, cudaStream_t st)
{
    TinyParams p{};
    p.in = in; p.out = out; p.m = s.m; p.n = s.n; p.steps = steps;
    p.ld = s.n | 1;   // odd: the rows' columns on different banks
    p.pairs = s.m * (s.m + 1) / 2;
    const int threads = s.m * s.n <= 512 ? 128 : 256;
    p.lanes = 1;
    while (p.lanes < 32 && p.pairs * p.lanes * 2 <= threads && p.lanes < s.n) p.lanes *= 2;
    for (int k = 0; k < 3 * steps; ++k) p.coeffs[k] = coeffs ? coeffs[k] : kNewtonCoeffs[k % 3];
    const size_t smem = (size_t)2 * kTinyRows * p.ld * sizeof(float);
    static bool attr[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GCONV_ERR_CUDA;
    if (!attr[dev]) {
        const int most = 2 * kTinyRows * (kTinyCols + 1) * (int)sizeof(float);
        if (cudaFuncSetAttribute(newton_tiny_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
            return GCONV_ERR_CUDA;
        attr[dev] = true;
    }
    launch_dependent(newton_tiny_kernel, (unsigned)s.G, threads, smem, st, p);
    return cudaGetLastError() == cudaSuccess ? GCONV_OK : GCONV_ERR_CUDA;
}

}  // namespace gconv
