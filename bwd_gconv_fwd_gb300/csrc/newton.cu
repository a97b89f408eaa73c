// newton.cu -- orthogonalisation of weight-shaped tensors by Newton-Schulz steps, and the
// Muon weight update built on it.  See include/gconv.h for the operations.
//
// A tensor [C_out][C_in/G][kH][kW] is G matrices.  Each is taken with its shorter side as
// rows (m <= n; a taller matrix is read and written transposed), scaled to unit Frobenius
// norm, and stepped: A = X X^T, P = a I + b A + c A A, X <- P X.  A and P are symmetric, so
// their tiles above the diagonal are mirrored, not computed: m^2 n + m^3 + 2 m^2 n
// operations a step.
//
// Precision.  X, A and P are kept in fp16 scaled by 2^8, products accumulate in fp32.
// Entries of X and A are at most about 1.2, so 2^8 keeps them below the largest fp16 with
// room for other coefficients, and entries down to 2^-22 normal.  A step multiplies the
// rounding of the step before by up to a = 3.44; with fp16's 11 bits the result is about 1e-3
// from the exact iteration (bf16's 8 bits: 1e-2), below the rounding of a bf16 result.
// Keeping a I inside P rather than adding a X afterwards rounds the difference a - |b| + c
// instead of its large terms.
#include "newton.cuh"

#include <cudaTypedefs.h>
#include <algorithm>
#include <climits>
#include <cmath>

namespace gconv {

namespace {

constexpr float kScale = kNewtonScale;
constexpr int kThreads = 352;     // warps 0, 6-10: TMA producers; 1: MMA; 2-5: epilogue
constexpr int kProducers = 6;
constexpr int kBM = 128, kBK = 64;
constexpr uint64_t kDrainNs = 1000000000ull;
constexpr int kNormBlocks = 64;   // partial sums of a matrix's squares, at most

enum { kGram = 0, kPoly = 1, kApply = 2 };

struct NewtonParams {
    int batch, M, N, K, ldc;
    int n_mblk, n_nblk, n_kblk, tiles_per, stages;
    __half *C;                   // gram: A, poly: P, apply: the next X (not the last step)
    const __half *A;             // poly: A
    float a, b, c;               // poly
    int last;
    NewtonOut o;
    unsigned int *err;
    uint64_t wait_ns;
};

// Sum over a block of 256 threads, in a fixed order; the result is in thread 0.
__device__ __forceinline__ float block_sum(float v, float *sh)
{
    #pragma unroll
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
    if (threadIdx.x < 32) {
        t = threadIdx.x < 8 ? sh[threadIdx.x] : 0.f;
        #pragma unroll
        for (int m = 4; m; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
    }
    return t;
}

// Updates the momentum and adds the squares of one share of one matrix.  grid (shares, G).
__global__ void __launch_bounds__(256) newton_norm_kernel(const NewtonIn p, float *part)
{
    __shared__ float sh[8];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t base = (int64_t)blockIdx.y * p.elems;
    float s = 0.f;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.elems; i += (int64_t)gridDim.x * 256) {
        float u = load_g(p, base + i);
        if (p.m) {
            const float m = fmaf(p.beta, p.m[base + i], u);
            p.m_out[base + i] = m;
            u = lookahead(p, u, m);
        }
        s = fmaf(u, u, s);
    }
    s = block_sum(s, sh);
    if (threadIdx.x == 0) part[blockIdx.y * kNormBlocks + blockIdx.x] = s;
}

// X = 2^8 u / (|u| + eps) in fp16, rows = the shorter side; 32 x 32 tiles of the matrix as it
// lies, through shared memory when it is transposed.  grid (column tiles, row tiles, G).
__global__ void __launch_bounds__(256) newton_scale_kernel(const NewtonIn p, const float *part, int parts, __half *x, int ldx)
{
    __shared__ float tile[32][33];
    __shared__ float inv_sh;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t base = (int64_t)blockIdx.z * p.elems;
    if (threadIdx.x < 32) {
        float s = 0.f;
        for (int i = threadIdx.x; i < parts; i += 32) s += part[blockIdx.z * kNormBlocks + i];
        #pragma unroll
        for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
        if (threadIdx.x == 0) inv_sh = kScale / (sqrtf(s) + p.eps);
    }
    __syncthreads();
    const float inv = inv_sh;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c0 = blockIdx.x * 32, r0 = blockIdx.y * 32;
    const int m_rows = p.tall ? p.cols : p.rows;
    for (int r = ty; r < 32; r += 8) {
        const int row = r0 + r, col = c0 + tx;
        float v = 0.f;
        if (row < p.rows && col < p.cols) {
            const int64_t i = base + (int64_t)row * p.cols + col;
            v = load_g(p, i);
            if (p.m) v = lookahead(p, v, p.m_out[i]);
            v *= inv;
            if (!p.tall) x[((int64_t)blockIdx.z * m_rows + row) * ldx + col] = __float2half_rn(v);
        }
        tile[r][tx] = v;
    }
    if (!p.tall) return;
    __syncthreads();
    for (int r = ty; r < 32; r += 8) {
        const int row = c0 + r, col = r0 + tx;   // of X
        if (row < p.cols && col < p.rows)
            x[((int64_t)blockIdx.z * m_rows + row) * ldx + col] = __float2half_rn(tile[tx][r]);
    }
}

// Tile t of the lower triangle, row by row: (row block, column block).
__device__ __forceinline__ void triangle(int t, int *mb, int *nb)
{
    int r = (int)((sqrtf(8.f * (float)t + 1.f) - 1.f) * 0.5f);
    while ((r + 1) * (r + 2) / 2 <= t) ++r;
    while (r * (r + 1) / 2 > t) --r;
    *mb = r;
    *nb = t - r * (r + 1) / 2;
}

// D = A B^T on 128 x BN tiles (gram, poly: both operands K-major, lower-triangle tiles only;
// apply: B = X is N-major).  Persistent CTAs; a ring of 64-deep stages filled by six TMA
// threads, one MMA thread, two accumulators so that four warps drain one while the other fills.
template <int BN, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
newton_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ NewtonParams p)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[8], bar_empty[8], bar_acc_full[2], bar_acc_empty[2], bar_drain;
    __shared__ uint32_t tmem_base_sh;
    __shared__ volatile int abort_flag;
    constexpr int b_mn = MODE == kApply ? 1 : 0;
    constexpr uint32_t tmem_cols = 2 * BN <= 256 ? 256u : 512u;
    constexpr uint32_t a_bytes = kBM * kBK * 2, b_bytes = BN * kBK * 2, stage_bytes = a_bytes + b_bytes;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sbase = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    const int n_tiles = p.batch * p.tiles_per;
    auto where = [&](int tile, int *bt, int *mb, int *nb) {
        *bt = tile / p.tiles_per;
        const int t = tile - *bt * p.tiles_per;
        if (MODE == kApply) { *mb = t % p.n_mblk; *nb = t / p.n_mblk; }
        else triangle(t, mb, nb);
    };

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < p.stages; ++i) {
            ptx::mbar_init(ptx::smem_u32(&bar_full[i]), kProducers);
            ptx::mbar_init(ptx::smem_u32(&bar_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_u32(&bar_acc_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&bar_acc_empty[i]), 128);
        }
        ptx::mbar_init(ptx::smem_u32(&bar_drain), 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tmA);
        ptx::prefetch_tmap(&tmB);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&tmem_base_sh), tmem_cols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    ptx::griddep_wait();
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();

    if (warp == 0 || warp >= 6) {
        // ---------------- TMA producers ----------------
        if (lane == 0) {
            const int pi = warp == 0 ? 0 : warp - 5;
            constexpr int nA = 2, nB = BN / 64;
            uint32_t my_bytes = 0;
            for (int i = pi; i < nA + nB; i += kProducers) my_bytes += 8192u;
            int it = 0;
            for (int tile = blockIdx.x; tile < n_tiles && !abort_flag; tile += gridDim.x) {
                int bt, mb, nb;
                where(tile, &bt, &mb, &nb);
                for (int kb = 0; kb < p.n_kblk && !abort_flag; ++kb, ++it) {
                    const int slot = it % p.stages;
                    if (it >= p.stages &&
                        !ptx::mbar_wait(ptx::smem_u32(&bar_empty[slot]), ((it / p.stages) - 1) & 1, p.wait_ns)) {
                        abort_flag = 1;
                        raise_device_error(p.err, DEVERR_WAIT_TIMEOUT);
                        break;
                    }
                    const uint32_t fb = ptx::smem_u32(&bar_full[slot]);
                    const uint32_t sa = sbase + slot * stage_bytes, sb = sa + a_bytes;
                    ptx::mbar_arrive_expect_tx(fb, my_bytes);
                    for (int i = pi; i < nA + nB; i += kProducers) {
                        if (i < nA) {
                            ptx::tma_load_3d(sa + i * 8192, &tmA, kb * kBK, mb * kBM + i * 64, bt, fb);
                        } else {
                            const int c = i - nA;
                            const int x = b_mn ? nb * BN + c * 64 : kb * kBK, y = b_mn ? kb * kBK : nb * BN + c * 64;
                            ptx::tma_load_3d(sb + c * 8192, &tmB, x, y, bt, fb);
                        }
                    }
                }
            }
            // drain: this thread's copies have landed once its last stages are full (bounded; after
            // an abort a stage may never fill, and the copies, issued long before, have landed)
            for (int j = max(0, it - p.stages); j < it; ++j)
                if (!ptx::mbar_wait(ptx::smem_u32(&bar_full[j % p.stages]), (j / p.stages) & 1, kDrainNs)) {
                    raise_device_error(p.err, DEVERR_WAIT_TIMEOUT);
                    break;
                }
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        if (lane == 0) {
            const uint32_t idesc = idesc_f16(kBM, BN, b_mn);
            const uint64_t a0 = ptx::smem_desc(sbase, 16, 1024, 2);
            const uint64_t b0 = b_mn ? ptx::smem_desc(sbase + a_bytes, 8192, 1024, 2)
                                     : ptx::smem_desc(sbase + a_bytes, 16, 1024, 2);
            constexpr uint64_t ak = 32 >> 4, bk = b_mn ? 2048 >> 4 : 32 >> 4;
            int local = 0, slot = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x, ++local) {
                const int buf = local & 1;
                if (local >= 2 && !ptx::mbar_test_wait(ptx::smem_u32(&bar_acc_empty[buf]), ((local >> 1) - 1) & 1))
                    ok = ptx::mbar_wait_ool(ptx::smem_u32(&bar_acc_empty[buf]), ((local >> 1) - 1) & 1, p.wait_ns, nullptr);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t dt = tmem + (uint32_t)(buf * BN);
                for (int kb = 0; kb < p.n_kblk; ++kb) {
                    const uint32_t fb = ptx::smem_u32(&bar_full[slot]);
                    if (!ptx::mbar_test_wait(fb, phase) && ok) ok = ptx::mbar_wait_ool(fb, phase, p.wait_ns, nullptr);
                    ptx::tc_fence_after();
                    const uint64_t so = (uint64_t)((slot * stage_bytes) >> 4);
                    const uint64_t ad = a0 + so, bd = b0 + so;
                    #pragma unroll
                    for (int k = 0; k < kBK / 16; ++k)
                        ptx::mma_f16(dt, ad + k * ak, bd + k * bk, idesc, (kb > 0 || k > 0) ? 1u : 0u);
                    ptx::mma_commit(ptx::smem_u32(&bar_empty[slot]));
                    if (++slot == p.stages) { slot = 0; phase ^= 1u; }
                }
                if (!ok) break;
                ptx::mma_commit(ptx::smem_u32(&bar_acc_full[buf]));
                if (abort_flag) ok = false;
            }
            if (!ok) {
                abort_flag = 1;
                raise_device_error(p.err, DEVERR_WAIT_TIMEOUT);
            }
        }
    } else {
        // ---------------- epilogue (warps 2-5 -> TMEM lane groups 2,3,0,1) ----------------
        const int lg = warp & 3;
        int local = 0;
        for (int tile = blockIdx.x; tile < n_tiles; tile += gridDim.x, ++local) {
            const int buf = local & 1;
            bool ready = ptx::mbar_wait(ptx::smem_u32(&bar_acc_full[buf]), (local >> 1) & 1, p.wait_ns);
            if (!ready) raise_device_error(p.err, DEVERR_WAIT_TIMEOUT);
            ready = __all_sync(0xffffffffu, ready && !abort_flag);
            if (!ready) break;
            ptx::tc_fence_after();
            int bt, mb, nb;
            where(tile, &bt, &mb, &nb);
            const int row = mb * kBM + lg * 32 + lane;
            __half *C = p.C + (int64_t)bt * p.M * p.ldc;
            const __half *A = MODE == kPoly ? p.A + (int64_t)bt * p.M * p.ldc : nullptr;
            for (int c0 = 0; c0 < BN; c0 += 16) {
                uint32_t acc[16];
                ptx::tmem_ld16(tmem + ((uint32_t)(lg * 32) << 16) + (uint32_t)(buf * BN + c0), acc);
                ptx::tmem_ld_wait();
                const int col0 = nb * BN + c0;
                if (row >= p.M || col0 >= p.N) continue;
                if (MODE == kApply) {
                    if (p.last) {
                        #pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (col0 + j < p.N)
                                store_result(p.o, (int64_t)bt * p.M * p.N + (p.o.tall ? (int64_t)(col0 + j) * p.M + row
                                                                                  : (int64_t)row * p.N + col0 + j),
                                             __uint_as_float(acc[j]) * (1.f / (kScale * kScale)));
                    } else {
                        __half2 h[8];
                        #pragma unroll
                        for (int j = 0; j < 8; ++j)
                            h[j] = __floats2half2_rn(__uint_as_float(acc[2 * j]) * (1.f / kScale),
                                                     __uint_as_float(acc[2 * j + 1]) * (1.f / kScale));
                        // rows are padded to 8 columns, which no product reads past N
                        uint4 *dst = reinterpret_cast<uint4 *>(C + (int64_t)row * p.ldc + col0);
                        dst[0] = *reinterpret_cast<uint4 *>(&h[0]);
                        if (col0 + 8 < p.N) dst[1] = *reinterpret_cast<uint4 *>(&h[4]);
                    }
                } else {
                    #pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int col = col0 + j;
                        float v = __uint_as_float(acc[j]) * (1.f / kScale);
                        if (col > row) continue;
                        if (MODE == kPoly) {
                            const float lin = __half2float(A[(int64_t)row * p.ldc + col]);
                            v = fmaf(p.c * (1.f), v, p.b * lin);
                            if (col == row) v += p.a * kScale;
                        }
                        const __half hv = __float2half_rn(v);
                        C[(int64_t)row * p.ldc + col] = hv;
                        if (col != row) C[(int64_t)col * p.ldc + row] = hv;
                    }
                }
            }
            ptx::tc_fence_before();
            ptx::mbar_arrive(ptx::smem_u32(&bar_acc_empty[buf]));
        }
    }
    if (warp == 1 && lane == 0) {
        ptx::mma_commit(ptx::smem_u32(&bar_drain));
        if (!ptx::mbar_wait(ptx::smem_u32(&bar_drain), 0, kDrainNs)) raise_device_error(p.err, DEVERR_WAIT_TIMEOUT);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) ptx::tmem_dealloc(tmem, tmem_cols);
}

// ---- host side ----------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
                cudaSuccess || q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// `batch` fp16 [rows][cols] matrices with rows ld elements apart, box 64 x 64, 128-byte swizzle.
bool half_tmap(CUtensorMap *m, const void *base, int cols, int rows, int ld, int batch)
{
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
    cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * rows * 2};
    cuuint32_t box[3] = {64u, 64u, 1u};
    cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

bool newton_shape(const gconv_matrices *t, NewtonShape *s)
{
    if (!t || t->rows < 1 || t->cols < 1 || t->count < 0) return false;
    const int64_t e = (int64_t)t->rows * t->cols;
    if (e > INT_MAX || e * t->count > INT_MAX) return false;
    s->G = t->count; s->rows = t->rows; s->cols = t->cols;
    s->tall = t->rows > t->cols;
    s->m = s->tall ? t->cols : t->rows;
    s->n = s->tall ? t->rows : t->cols;
    s->ldx = (s->n + 7) & ~7;
    s->lda = (s->m + 7) & ~7;
    s->x_bytes = up256((size_t)s->G * s->m * s->ldx * 2);
    s->a_bytes = up256((size_t)s->G * s->m * s->lda * 2);
    s->ws = up256((size_t)s->G * kNormBlocks * 4) + 2 * s->x_bytes + 2 * s->a_bytes;
    return true;
}

constexpr size_t kMaxSmem = 220 * 1024;

template <int BN, int MODE>
gconv_status launch_gemm(const CUtensorMap &tA, const CUtensorMap &tB, NewtonParams p, cudaStream_t st)
{
    p.n_mblk = (p.M + kBM - 1) / kBM;
    p.n_nblk = (p.N + BN - 1) / BN;
    p.n_kblk = (p.K + kBK - 1) / kBK;
    p.tiles_per = MODE == kApply ? p.n_mblk * p.n_nblk : p.n_mblk * (p.n_mblk + 1) / 2;
    const size_t stage = (size_t)(kBM + BN) * kBK * 2;
    p.stages = (int)std::min<size_t>(8, (kMaxSmem - 1024) / stage);
    static bool attr[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GCONV_ERR_CUDA;
    if (!attr[dev]) {
        if (cudaFuncSetAttribute(newton_gemm_kernel<BN, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)kMaxSmem) != cudaSuccess)
            return GCONV_ERR_CUDA;
        attr[dev] = true;
    }
    const int64_t tiles = (int64_t)p.batch * p.tiles_per;
    launch_dependent(newton_gemm_kernel<BN, MODE>, (unsigned)std::min<int64_t>(tiles, num_sms()), kThreads,
                     p.stages * stage + 1024, st, tA, tB, p);
    return GCONV_OK;
}

gconv_status run_newton(const NewtonShape &s, NewtonIn in, const NewtonOut &out, int steps, const float *coeffs,
                        void *workspace, cudaStream_t st)
{
    unsigned int *err = device_error_word();
    if (!err) return GCONV_ERR_CUDA;
    cudaGetLastError();   // clear a stale error: the check after the launches is about this call
    NewtonOut o = out;
    o.tall = in.tall = s.tall; in.rows = s.rows; in.cols = s.cols; in.elems = (int64_t)s.rows * s.cols;
    if (newton_small_fits(s)) return newton_small_launch(s, in, o, steps, coeffs, err, st);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    float *part = reinterpret_cast<float *>(ws);
    ws += up256((size_t)s.G * kNormBlocks * 4);
    __half *x[2] = {reinterpret_cast<__half *>(ws), reinterpret_cast<__half *>(ws + s.x_bytes)};
    ws += 2 * s.x_bytes;
    __half *A = reinterpret_cast<__half *>(ws), *P = reinterpret_cast<__half *>(ws + s.a_bytes);
    CUtensorMap tX[2], tA, tP;
    if (!half_tmap(&tX[0], x[0], s.n, s.m, s.ldx, s.G) || !half_tmap(&tX[1], x[1], s.n, s.m, s.ldx, s.G) ||
        !half_tmap(&tA, A, s.m, s.m, s.lda, s.G) || !half_tmap(&tP, P, s.m, s.m, s.lda, s.G))
        return GCONV_ERR_CUDA;
    const int parts = (int)std::min<int64_t>(kNormBlocks, (in.elems + 1023) / 1024);
    for (int g0 = 0; g0 < s.G; g0 += 65535) {   // grid y and z are 16 bits
        const int g = std::min(65535, s.G - g0);
        NewtonIn part_in = in;
        const int64_t off = (int64_t)g0 * in.elems;
        part_in.g = static_cast<const uint8_t *>(in.g) + off * (in.g_bf16 ? 2 : 4);
        if (in.m) { part_in.m = in.m + off; part_in.m_out = in.m_out + off; }
        newton_norm_kernel<<<dim3(parts, g), 256, 0, st>>>(part_in, part + (size_t)g0 * kNormBlocks);
        newton_scale_kernel<<<dim3((s.cols + 31) / 32, (s.rows + 31) / 32, g), 256, 0, st>>>(
            part_in, part + (size_t)g0 * kNormBlocks, parts, x[0] + (int64_t)g0 * s.m * s.ldx, s.ldx);
    }
    for (int k = 0; k < steps; ++k) {
        const float *c = coeffs ? coeffs + 3 * k : kNewtonCoeffs;
        NewtonParams p{};
        p.batch = s.G; p.err = err; p.wait_ns = (uint64_t)wait_limit();
        p.M = s.m; p.N = s.m; p.K = s.n; p.ldc = s.lda; p.C = A;
        gconv_status r = launch_gemm<128, kGram>(tX[k & 1], tX[k & 1], p, st);
        if (r != GCONV_OK) return r;
        p.K = s.m; p.C = P; p.A = A;
        p.a = c[0]; p.b = c[1]; p.c = c[2];
        r = launch_gemm<128, kPoly>(tA, tA, p, st);
        if (r != GCONV_OK) return r;
        p.N = s.n; p.ldc = s.ldx; p.C = x[(k + 1) & 1];
        p.last = k + 1 == steps;
        p.o = o;
        r = launch_gemm<256, kApply>(tP, tX[k & 1], p, st);
        if (r != GCONV_OK) return r;
    }
    return cudaGetLastError() == cudaSuccess ? GCONV_OK : GCONV_ERR_CUDA;
}

bool good(float v) { return v == v && v <= 3e38f && v >= -3e38f; }

bool good_steps(int steps, const float *coeffs, float eps)
{
    if (steps < 1 || steps > kNewtonSteps || !good(eps) || eps < 0.f) return false;
    for (int i = 0; coeffs && i < 3 * steps; ++i)
        if (!good(coeffs[i])) return false;
    return true;
}

}  // namespace

}  // namespace gconv

using namespace gconv;

extern "C" {

size_t gconv_orthogonalize_workspace_size(const gconv_matrices *matrices)
{
    NewtonShape s;
    return newton_shape(matrices, &s) ? (s.G ? s.ws : 0) : (size_t)-1;
}

gconv_status gconv_orthogonalize(const gconv_matrices *matrices, gconv_dtype dtype, gconv_dtype out_dtype, const void *g,
                                 void *out, int steps, const float *coeffs, float eps, void *workspace,
                                 size_t workspace_bytes, void *stream)
{
    NewtonShape s;
    if (!newton_shape(matrices, &s) || !good_steps(steps, coeffs, eps)) return GCONV_ERR_INVALID_ARG;
    if ((dtype != GCONV_F32 && dtype != GCONV_BF16) || (out_dtype != GCONV_F32 && out_dtype != GCONV_BF16))
        return GCONV_ERR_INVALID_ARG;
    if (s.G == 0) return GCONV_OK;
    if (!g || !out || !aligned16(g) || !aligned16(out) || !aligned16(workspace)) return GCONV_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < s.ws) return GCONV_ERR_WORKSPACE;
    NewtonIn in{};
    in.g = g; in.g_bf16 = dtype == GCONV_BF16; in.eps = eps;
    NewtonOut o{};
    o.out = out; o.out_bf16 = out_dtype == GCONV_BF16;
    return run_newton(s, in, o, steps, coeffs, workspace, static_cast<cudaStream_t>(stream));
}

gconv_status gconv_muon_step(const gconv_matrices *matrices, const gconv_muon *opt, const float *w, const float *grad,
                             const float *momentum, float *w_out, float *momentum_out, void *w_bf16, void *workspace,
                             size_t workspace_bytes, void *stream)
{
    NewtonShape s;
    if (!newton_shape(matrices, &s) || !opt || !good_steps(opt->steps, opt->coeffs, opt->eps)) return GCONV_ERR_INVALID_ARG;
    if (!good(opt->lr) || !good(opt->beta) || !good(opt->weight_decay) || !good(opt->scale)) return GCONV_ERR_INVALID_ARG;
    if (s.G == 0) return GCONV_OK;
    if (!w || !grad || !momentum || !w_out || !momentum_out) return GCONV_ERR_INVALID_ARG;
    for (const void *q : {(const void *)w, (const void *)grad, (const void *)momentum, (const void *)w_out,
                          (const void *)momentum_out, (const void *)w_bf16, (const void *)workspace})
        if (!aligned16(q)) return GCONV_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < s.ws) return GCONV_ERR_WORKSPACE;
    NewtonIn in{};
    in.g = grad; in.m = momentum; in.m_out = momentum_out; in.beta = opt->beta; in.nesterov = opt->nesterov != 0;
    in.eps = opt->eps;
    NewtonOut o{};
    o.muon = 1; o.w = w; o.w_out = w_out; o.w_bf16 = static_cast<__nv_bfloat16 *>(w_bf16);
    o.keep = 1.f - opt->lr * opt->weight_decay;
    const float scale = opt->scale > 0.f ? opt->scale : std::sqrt(std::max(1.f, (float)s.rows / (float)s.cols));
    o.rate = opt->lr * scale;
    return run_newton(s, in, o, opt->steps, opt->coeffs, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
