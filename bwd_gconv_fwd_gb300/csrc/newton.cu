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
//
// Which kernels.  At most 16 x 1024 with m m n <= 32768: one block a matrix, fp32 (newton_tiny.cu).  A
// shorter side of at most 128 that a cluster's shared memory holds: one launch (newton_small.cu).
// Else, here, three or four launches a step, as programmatic dependents.  Five steps of 64 x 576 81 us
// by this file's products and 24 in a cluster, of 128 x 4096 113 and 53.
//   4096 x 9216 (a fully connected layer), 2663 GFLOP: 1.73 to 2.0 ms, 1.3 to 1.5 PFLOP/s of the 1.9 of a
// library product; the tensor cores are the limit (the power cap, when hot).  A Muon step of 1024 x
// 4608, 78 GFLOP: 225 us, 0.35 PFLOP/s; 22 launches of 7 to 16 us, of which a pipeline's start and drain
// are most.
#include "newton.cuh"

#include <cudaTypedefs.h>
#include <algorithm>
#include <climits>
#include <cmath>

namespace gconv {

namespace {

constexpr float kScale = kNewtonScale;
constexpr int kTile = 256;         // a pair of CTAs computes 256 x 256, 128 rows each
constexpr int kBK = 64;
constexpr int kStages = 6;
constexpr uint32_t kOperand = 128 * kBK * 2, kStageBytes = 2 * kOperand;   // one CTA's half of A and of B
constexpr int kProducers = 4, kDrainers = 8;
constexpr int kThreads = 32 * (1 + kProducers + kDrainers);
constexpr int kStagePitch = 33;    // floats of a staged row
constexpr uint32_t kWarpStage = 32 * kStagePitch * 4;
constexpr uint32_t kSmem = 1024 + kStages * kStageBytes + kDrainers * kWarpStage;
constexpr uint64_t kDrainNs = 1000000000ull;
constexpr int kNormBlocks = 1024;  // partial sums of a matrix's squares, at most
constexpr int kNormShare = 8192;   // elements of one

enum { kGram = 0, kPoly = 1, kApply = 2 };

struct NewtonParams {
    int batch, M, N, K, ldc;
    int n_mblk, n_kblk, tiles_per, splits, k_per;
    __half *C;                   // gram: A, poly: P, apply: the next X (not the last step)
    const __half *A;             // poly: A
    float *part;                 // gram in several splits: their sums
    float a, b, c;               // poly
    int last;
    NewtonOut o;
    unsigned int *err;
    uint64_t wait_ns;
};

// ---- norm and scale -------------------------------------------------------------

template <int V>
__device__ __forceinline__ void load_v(const float *p, int64_t i, float (&v)[V])
{
    #pragma unroll
    for (int k = 0; k < V; k += 4) {
        if constexpr (V >= 4) {
            const float4 q = *reinterpret_cast<const float4 *>(p + i + k);
            v[k] = q.x; v[k + 1] = q.y; v[k + 2] = q.z; v[k + 3] = q.w;
        } else {
            v[k] = p[i + k];
        }
    }
}

template <int V>
__device__ __forceinline__ void load_gv(const NewtonIn &p, int64_t i, float (&v)[V])
{
    if constexpr (V == 8) {
        if (p.g_bf16) {
            const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.g) + i);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
            #pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[2 * k] = __uint_as_float(w[k] << 16);
                v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            }
            return;
        }
        load_v<V>(static_cast<const float *>(p.g), i, v);
    } else {
        v[0] = load_g(p, i);
    }
}

// Updates the momentum and adds the squares of one share of one matrix.  grid (shares, G); bound by
// the memory (1024 x 4608 fp32, 57 MB read and written: 9.5 us).
// V = 8 where a matrix is a multiple of eight elements.
template <int V>
__global__ void __launch_bounds__(256) newton_norm_kernel(const NewtonIn p, float *part, int64_t share)
{
    __shared__ float sh[8];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t base = (int64_t)blockIdx.y * p.elems;
    const int64_t i0 = (int64_t)blockIdx.x * share, i1 = min(i0 + share, p.elems);
    float s = 0.f;
    #pragma unroll 4
    for (int64_t i = i0 + (int64_t)threadIdx.x * V; i < i1; i += 256 * V) {
        float u[V];
        load_gv<V>(p, base + i, u);
        if (p.m) {
            float m[V];
            load_v<V>(p.m, base + i, m);
            #pragma unroll
            for (int k = 0; k < V; ++k) {
                m[k] = fmaf(p.beta, m[k], u[k]);
                u[k] = lookahead(p, u[k], m[k]);
            }
            #pragma unroll
            for (int k = 0; k < V; k += 4) {
                if constexpr (V == 8) *reinterpret_cast<float4 *>(p.m_out + base + i + k) = make_float4(m[k], m[k + 1], m[k + 2], m[k + 3]);
                else p.m_out[base + i] = m[0];
            }
        }
        #pragma unroll
        for (int k = 0; k < V; ++k) s = fmaf(u[k], u[k], s);
    }
    #pragma unroll
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        float t = 0.f;
        for (int k = 0; k < 8; ++k) t += sh[k];
        part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = t;
    }
}

// 2^8 / (|u| + eps) from a matrix's shares, in a fixed order, for a block of 256 threads.
__device__ __forceinline__ float inverse_norm(const float *part, int parts, float eps, float *sh)
{
    float s = 0.f;
    for (int i = threadIdx.x; i < parts; i += 256) s += part[i];
    #pragma unroll
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
    __syncthreads();
    float t = 0.f;
    for (int k = 0; k < 8; ++k) t += sh[k];
    return unit_factor(kScale, t, eps);
}

// X = 2^8 u / (|u| + eps) in fp16 for matrices as wide as X and a multiple of eight columns:
// grid (shares, G), eight elements a thread; the memory is the limit (1024 x 4608: 10 us, cold).
__global__ void __launch_bounds__(256) newton_scale_flat_kernel(const NewtonIn p, const float *part, int parts, __half *x)
{
    __shared__ float sh[8];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const float inv = inverse_norm(part + (int64_t)blockIdx.y * parts, parts, p.eps, sh);
    const int64_t base = (int64_t)blockIdx.y * p.elems;
    const int64_t i0 = (int64_t)blockIdx.x * kNormShare, i1 = min(i0 + kNormShare, p.elems);
    #pragma unroll 4
    for (int64_t i = i0 + (int64_t)threadIdx.x * 8; i < i1; i += 256 * 8) {
        float u[8];
        load_gv<8>(p, base + i, u);
        if (p.m) {
            float m[8];
            load_v<8>(p.m_out, base + i, m);
            #pragma unroll
            for (int k = 0; k < 8; ++k) u[k] = lookahead(p, u[k], m[k]);
        }
        uint32_t h[4];
        #pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = half2_bits(u[2 * k] * inv, u[2 * k + 1] * inv);
        *reinterpret_cast<uint4 *>(x + base + i) = make_uint4(h[0], h[1], h[2], h[3]);
    }
}

// The same for any matrix: 64 x 32 tiles of the matrix as it lies, through shared memory when
// X is its transpose.  grid (column tiles x row tiles, G).
__global__ void __launch_bounds__(256) newton_scale_kernel(const NewtonIn p, const float *part, int parts, __half *x, int ldx,
                                                           int col_tiles)
{
    __shared__ float tile[64][33];
    __shared__ float sh[8];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const float inv = inverse_norm(part + (int64_t)blockIdx.y * parts, parts, p.eps, sh);
    const int64_t base = (int64_t)blockIdx.y * p.elems;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c0 = (int)(blockIdx.x % col_tiles) * 32, r0 = (int)(blockIdx.x / col_tiles) * 64;
    const int m_rows = p.tall ? p.cols : p.rows;
    __half *xb = x + (int64_t)blockIdx.y * m_rows * ldx;
    float v[8];
    #pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int row = r0 + ty + 8 * k, col = c0 + tx;
        v[k] = 0.f;
        if (row < p.rows && col < p.cols) {
            const int64_t i = base + (int64_t)row * p.cols + col;
            v[k] = load_g(p, i);
            if (p.m) v[k] = lookahead(p, v[k], p.m_out[i]);
            v[k] *= inv;
        }
    }
    if (!p.tall) {
        #pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int row = r0 + ty + 8 * k, col = c0 + tx;
            if (row < p.rows && col < p.cols) xb[(int64_t)row * ldx + col] = __float2half_rn(v[k]);
        }
        return;
    }
    #pragma unroll
    for (int k = 0; k < 8; ++k) tile[ty + 8 * k][tx] = v[k];
    __syncthreads();
    // two neighbouring columns of X a thread: ldx is a multiple of eight, so the second is in bounds
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int row = c0 + ty + 8 * k, col = r0 + 2 * tx;
        if (row < p.cols && col < p.rows)
            *reinterpret_cast<uint32_t *>(xb + (int64_t)row * ldx + col) =
                half2_bits(tile[2 * tx][ty + 8 * k], tile[2 * tx + 1][ty + 8 * k]);
    }
}

// ---- products ---------------------------------------------------------------------

// Tile t of the lower triangle, row by row, of tiles of 256 rows and BN columns: (row block,
// column block).  Row block r has (r + 1) 256 / BN tiles, those of its diagonal block included.
template <int BN>
__device__ __forceinline__ void triangle(int t, int *mb, int *nb)
{
    constexpr int per = kTile / BN;
    int r = (int)((sqrtf(8.f * (float)(t / per) + 1.f) - 1.f) * 0.5f);
    while (per * (r + 1) * (r + 2) / 2 <= t) ++r;
    while (per * r * (r + 1) / 2 > t) --r;
    *mb = r;
    *nb = t - per * r * (r + 1) / 2;
}

// A 32 x 32 block of a symmetric result: lane = row r0 + lane, v its 32 columns from c0.
// Rows are ldc (a multiple of eight) elements; columns M..ldc get zeros.
__device__ __forceinline__ void store_symmetric(__half *C, int M, int ldc, int r0, int c0, const float (&v)[32],
                                                bool mirror, __half *stage, int lane)
{
    uint32_t h[16];
    #pragma unroll
    for (int j = 0; j < 16; ++j) h[j] = half2_bits(v[2 * j], v[2 * j + 1]);
    const int row = r0 + lane;
    if (row < M) {
        #pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c0 + 8 * j < M)
                *reinterpret_cast<uint4 *>(C + (int64_t)row * ldc + c0 + 8 * j) =
                    make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
    }
    if (!mirror) return;
    constexpr int pitch = 40;   // halves: 16-byte rows, lanes of one column on neighbouring banks
    #pragma unroll
    for (int j = 0; j < 16; ++j) {
        const __half2 hh = *reinterpret_cast<const __half2 *>(&h[j]);
        stage[(2 * j) * pitch + lane] = __low2half(hh);
        stage[(2 * j + 1) * pitch + lane] = __high2half(hh);
    }
    __syncwarp();
    #pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int col = j * 8 + (lane >> 2), part = (lane & 3) * 8;
        if (c0 + col < M && r0 + part < M)
            *reinterpret_cast<uint4 *>(C + (int64_t)(c0 + col) * ldc + r0 + part) =
                *reinterpret_cast<const uint4 *>(stage + col * pitch + part);
    }
    __syncwarp();
}

// D = A B^T on 256 x BN tiles by pairs of CTAs (gram, poly: both operands K-major, lower
// triangle only; apply: B = X is N-major).  Each CTA holds 128 rows of A and 128 columns of
// B, so a stage is 32 KB a CTA for 2 x 2^21 products: a CTA alone with a 128 x 256 tile loads
// half as much again, and the loads, not the tensor cores, were its limit.  Persistent pairs; a
// ring of 64-deep stages filled by four TMA threads a CTA, one MMA thread a pair, two
// accumulators so that eight warps a CTA drain one while the other fills.  BN = 128 where 256
// would leave half the pairs without a tile: the fill and the drain of one tile are then the time.
template <int MODE, int BN>
__global__ void __launch_bounds__(kThreads, 1)
newton_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ NewtonParams p)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[kStages], bar_empty[kStages], bar_nobody[kStages], bar_acc_full[2], bar_acc_empty[2], bar_drain;
    __shared__ uint32_t tmem_base_sh;
    __shared__ volatile int abort_flag;
    constexpr int b_mn = MODE == kApply ? 1 : 0;
    constexpr int boxes = 2 + BN / 128;                     // 8 KB boxes of a stage and CTA
    constexpr int blocks = BN / 64;                         // 32-column blocks a drain warp

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_rank();
    const uint32_t sbase = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    const int units = p.batch * p.tiles_per * p.splits;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    auto where = [&](int u, int *bt, int *mb, int *nb, int *k0, int *k1) {
        const int sp = u % p.splits, tile = u / p.splits;
        *bt = tile / p.tiles_per;
        const int t = tile - *bt * p.tiles_per;
        if (MODE == kApply) { *mb = t % p.n_mblk; *nb = t / p.n_mblk; }
        else triangle<BN>(t, mb, nb);
        *k0 = sp * p.k_per;
        *k1 = min(p.n_kblk, *k0 + p.k_per);
    };

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(ptx::smem_u32(&bar_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&bar_empty[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&bar_nobody[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_u32(&bar_acc_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&bar_acc_empty[i]), 2 * kDrainers);
        }
        ptx::mbar_init(ptx::smem_u32(&bar_drain), 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tmA);
        ptx::prefetch_tmap(&tmB);
    }
    if (warp == 0) {
        tmem_alloc_pair(ptx::smem_u32(&tmem_base_sh), 512);
        tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    ptx::griddep_wait();
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();

    if (warp >= 1 && warp <= kProducers) {
        // ---------------- TMA producers: one 8 KB box a stage each ----------------
        if (lane == 0 && warp - 1 < boxes) {
            const int pi = warp - 1;                        // 0, 1: halves of A; 2, 3: B
            int it = 0;
            for (int u = pair; u < units && !abort_flag; u += pairs) {
                int bt, mb, nb, k0, k1;
                where(u, &bt, &mb, &nb, &k0, &k1);
                const int r = pi < 2 ? mb * kTile + (int)rank * 128 + pi * 64 : nb * BN + (int)rank * (BN / 2) + (pi - 2) * 64;
                for (int kb = k0; kb < k1 && !abort_flag; ++kb, ++it) {
                    const int slot = it % kStages;
                    if (it >= kStages &&
                        !ptx::mbar_wait(ptx::smem_u32(&bar_empty[slot]), ((it / kStages) - 1) & 1, p.wait_ns)) {
                        abort_flag = 1;
                        raise_device_error(p.err, DEVERR_WAIT_TIMEOUT);
                        break;
                    }
                    // the pair's stage is one barrier in the first CTA
                    const uint32_t local = ptx::smem_u32(&bar_full[slot]);
                    if (rank == 0 && pi == 0) ptx::mbar_arrive_expect_tx(local, 2 * boxes * 8192);
                    const uint32_t fb = ptx::map_to(local, 0);
                    const uint32_t dst = sbase + slot * kStageBytes + pi * 8192;
                    if (pi >= 2 && b_mn) tma_load_pair(dst, &tmB, r, kb * kBK, bt, fb);
                    else tma_load_pair(dst, pi < 2 ? &tmA : &tmB, kb * kBK, r, bt, fb);
                }
            }
            // drain: the copies of the last stages have been consumed once their slots are free
            for (int j = max(0, it - kStages); j < it; ++j)
                if (!ptx::mbar_wait(ptx::smem_u32(&bar_empty[j % kStages]), (j / kStages) & 1, kDrainNs)) {
                    raise_device_error(p.err, DEVERR_WAIT_TIMEOUT);
                    break;
                }
        }
    } else if (warp == 0) {
        // ---------------- MMA issuer of the pair ----------------
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = idesc_f16(kTile, BN, b_mn);
            const uint64_t a0 = ptx::smem_desc(sbase, 16, 1024, 2);
            const uint64_t b0 = b_mn ? ptx::smem_desc(sbase + kOperand, 8192, 1024, 2)
                                     : ptx::smem_desc(sbase + kOperand, 16, 1024, 2);
            constexpr uint64_t ak = 32 >> 4, bk = b_mn ? 2048 >> 4 : 32 >> 4;
            int local = 0, slot = 0;
            uint32_t phase = 0;
            bool ok = true;
            // After a wait that gave up no slot is handed back, as it would be filled while its phase may
            // be open: the rest of the unit signals barriers that nobody waits for.  (Leaving the loop there
            // made its code slower: 4096 x 9216 2010 us against 1953.)
            uint32_t empties = ptx::smem_u32(bar_empty);
            for (int u = pair; u < units && ok; u += pairs, ++local) {
                int bt, mb, nb, k0, k1;
                where(u, &bt, &mb, &nb, &k0, &k1);
                const int buf = local & 1;
                if (local >= 2 && !ptx::mbar_test_wait(ptx::smem_u32(&bar_acc_empty[buf]), ((local >> 1) - 1) & 1))
                    ok = ptx::mbar_wait_ool(ptx::smem_u32(&bar_acc_empty[buf]), ((local >> 1) - 1) & 1, p.wait_ns, nullptr);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t dt = tmem + (uint32_t)(buf * BN);
                for (int kb = k0; kb < k1; ++kb) {
                    const uint32_t fb = ptx::smem_u32(&bar_full[slot]);
                    if (!ptx::mbar_test_wait(fb, phase) && ok) {
                        ok = ptx::mbar_wait_ool(fb, phase, p.wait_ns, nullptr);
                        if (!ok) empties = ptx::smem_u32(bar_nobody);
                    }
                    ptx::tc_fence_after();
                    const uint64_t so = (uint64_t)((slot * kStageBytes) >> 4);
                    const uint64_t ad = a0 + so, bd = b0 + so;
                    #pragma unroll
                    for (int k = 0; k < kBK / 16; ++k)
                        mma_f16_pair(dt, ad + k * ak, bd + k * bk, idesc, (kb > k0 || k > 0) ? 1u : 0u);
                    mma_commit_pair(empties + 8u * (uint32_t)slot);
                    if (++slot == kStages) { slot = 0; phase ^= 1u; }
                }
                if (!ok) break;
                mma_commit_pair(ptx::smem_u32(&bar_acc_full[buf]));
                if (abort_flag) ok = false;
            }
            if (!ok) {
                abort_flag = 1;
                raise_device_error(p.err, DEVERR_WAIT_TIMEOUT);
            }
        }
    } else {
        // ---------------- drain: lanes 32 lg.. of tensor memory, half the columns a warp ----------------
        const int lg = warp & 3, dw = warp - 1 - kProducers;
        const int half = dw >> 2;
        uint8_t *stage8 = smem_raw + (sbase - ptx::smem_u32(smem_raw)) + kStages * kStageBytes + dw * kWarpStage;
        float *stage = reinterpret_cast<float *>(stage8);
        int local = 0;
        for (int u = pair; u < units; u += pairs, ++local) {
            const int buf = local & 1;
            int bt, mb, nb, k0, k1;
            where(u, &bt, &mb, &nb, &k0, &k1);
            const int r0 = mb * kTile + (int)rank * 128 + lg * 32, row = r0 + lane;
            __half *C = p.C + (int64_t)bt * p.M * p.ldc;
            const int64_t out0 = (int64_t)bt * p.M * p.N;
            // What a block needs from memory beside the product is read a block ahead, the first
            // before the product is done: A's elements (poly), the weights (Muon's last step).
            uint4 lin[4];
            float wv[32];
            const bool weights = MODE == kApply && p.last && p.o.muon && !p.o.tall;
            auto ahead = [&](int blk) {
                const int c0 = nb * BN + blk * 32;
                if constexpr (MODE == kPoly) {
                    const __half *A = p.A + (int64_t)bt * p.M * p.ldc + (int64_t)row * p.ldc + c0;
                    #pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        lin[j] = make_uint4(0, 0, 0, 0);
                        if (row < p.M && c0 + 8 * j < p.M) lin[j] = *reinterpret_cast<const uint4 *>(A + 8 * j);
                    }
                }
                if constexpr (MODE == kApply) {
                    if (weights) {
                        #pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (r0 + j < p.M && c0 + lane < p.N) wv[j] = p.o.w[out0 + (int64_t)(r0 + j) * p.N + c0 + lane];
                    }
                }
            };
            ahead(half * blocks);
            bool ready = ptx::mbar_wait(ptx::smem_u32(&bar_acc_full[buf]), (local >> 1) & 1, p.wait_ns);
            if (!ready) raise_device_error(p.err, DEVERR_WAIT_TIMEOUT);
            ready = __all_sync(0xffffffffu, ready && !abort_flag);
            if (!ready) break;
            ptx::tc_fence_after();
            for (int blk = half * blocks; blk < half * blocks + blocks; ++blk) {
                uint32_t raw[2][16];
                const uint32_t at = tmem + ((uint32_t)(lg * 32) << 16) + (uint32_t)(buf * BN + blk * 32);
                ptx::tmem_ld16(at, raw[0]);
                ptx::tmem_ld16(at + 16, raw[1]);
                ptx::tmem_ld_wait();
                const int c0 = nb * BN + blk * 32;
                if (r0 >= p.M || c0 >= p.N) continue;
                float v[32];
                #pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j >> 4][j & 15]);
                if (MODE == kGram && p.splits > 1) {
                    // [unit][CTA][drain warp][block][4 columns][lane]: newton_sum_kernel reads it the same way
                    float4 *dst = reinterpret_cast<float4 *>(p.part) +
                                  ((((int64_t)u * 2 + rank) * kDrainers + dw) * blocks + (blk - half * blocks)) * 256 + lane;
                    #pragma unroll
                    for (int j = 0; j < 8; ++j)
                        dst[j * 32] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                } else if (MODE == kGram) {
                    #pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] *= 1.f / kScale;
                    store_symmetric(C, p.M, p.ldc, r0, c0, v, mb != nb * BN / kTile, reinterpret_cast<__half *>(stage8), lane);
                } else if (MODE == kPoly) {
                    #pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t w[4] = {lin[j].x, lin[j].y, lin[j].z, lin[j].w};
                        #pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 l = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
                            v[8 * j + 2 * k] = fmaf(p.c * (1.f / kScale), v[8 * j + 2 * k], p.b * l.x);
                            v[8 * j + 2 * k + 1] = fmaf(p.c * (1.f / kScale), v[8 * j + 2 * k + 1], p.b * l.y);
                        }
                    }
                    if (blk + 1 < half * blocks + blocks) ahead(blk + 1);
                    if (r0 == c0) {
                        #pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j == lane && row < p.M) v[j] += p.a * kScale;
                    }
                    store_symmetric(C, p.M, p.ldc, r0, c0, v, mb != nb * BN / kTile, reinterpret_cast<__half *>(stage8), lane);
                } else if (!p.last) {
                    if (row < p.M) {
                        #pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t h[4];
                            #pragma unroll
                            for (int k = 0; k < 4; ++k)
                                h[k] = half2_bits(v[8 * j + 2 * k] * (1.f / kScale), v[8 * j + 2 * k + 1] * (1.f / kScale));
                            // rows are padded to eight columns, which no product reads past N
                            if (c0 + 8 * j < p.N)
                                *reinterpret_cast<uint4 *>(C + (int64_t)row * p.ldc + c0 + 8 * j) =
                                    make_uint4(h[0], h[1], h[2], h[3]);
                        }
                    }
                } else {
                    constexpr float back = 1.f / (kScale * kScale);
                    if (p.o.tall) {
                        #pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (row < p.M && c0 + j < p.N) store_result(p.o, out0 + (int64_t)(c0 + j) * p.M + row, v[j] * back);
                    } else {
                        #pragma unroll
                        for (int j = 0; j < 32; ++j) stage[lane * kStagePitch + j] = v[j] * back;
                        __syncwarp();
                        const int64_t at0 = out0 + (int64_t)r0 * p.N + c0 + lane;
                        float res[32];
                        #pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            res[j] = stage[j * kStagePitch + lane];
                            if (weights) res[j] = fmaf(-p.o.rate, res[j], p.o.keep * wv[j]);
                        }
                        if (blk + 1 < half * blocks + blocks) ahead(blk + 1);
                        #pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (r0 + j < p.M && c0 + lane < p.N) put_result(p.o, at0 + (int64_t)j * p.N, res[j]);
                        __syncwarp();
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_at(ptx::smem_u32(&bar_acc_empty[buf]), 0);
        }
    }
    if (warp == 0 && lane == 0 && rank == 0) {
        // every issued MMA ends before tensor memory is released
        mma_commit_pair_here(ptx::smem_u32(&bar_drain));
        if (!ptx::mbar_wait(ptx::smem_u32(&bar_drain), 0, kDrainNs)) raise_device_error(p.err, DEVERR_WAIT_TIMEOUT);
    }
    __syncwarp();
    ptx::tc_fence_before();
    ptx::cluster_sync();   // no CTA leaves while the other may signal it or use its operands
    if (warp == 0) tmem_dealloc_pair(tmem, 512);
}

// A = the sum of the splits of a gram, in split order, scaled, rounded and mirrored.  A warp
// takes 32 rows x 8 columns of a tile, so that all its loads are in flight at once (1024 rows in seven
// splits, 18 MB of fp32 out of L2: 7.5 us alone).
template <int BN>
__global__ void __launch_bounds__(256) newton_sum_kernel(const __grid_constant__ NewtonParams p)
{
    constexpr int pitch = 40;
    __shared__ __align__(16) __half stage[8][8 * pitch];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    constexpr int blocks = BN / 64;                        // of 32 columns a drain warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = blockIdx.x * 8 + warp;
    const int quarter = w & 3, b = (w >> 2) % blocks, dw = (w >> 2) / blocks & 7, rank = (w >> 2) / (blocks * 8) & 1;
    const int tile = (w >> 2) / (blocks * 16);
    if (tile >= p.batch * p.tiles_per) return;
    const int bt = tile / p.tiles_per;
    int mb, nb;
    triangle<BN>(tile - bt * p.tiles_per, &mb, &nb);
    const int lg = (dw + 1 + kProducers) & 3, blk = (dw >> 2) * blocks + b;
    const int r0 = mb * kTile + rank * 128 + lg * 32, c0 = nb * BN + blk * 32 + quarter * 8;
    if (r0 >= p.M || c0 >= p.N) return;
    float v[8] = {};
    const float4 *src = reinterpret_cast<const float4 *>(p.part) +
                        ((((int64_t)tile * p.splits * 2 + rank) * kDrainers + dw) * blocks + b) * 256 + quarter * 64 + lane;
    const int64_t hop = (int64_t)2 * kDrainers * blocks * 256;
    #pragma unroll 8
    for (int s = 0; s < p.splits; ++s) {
        const float4 x = src[s * hop], y = src[s * hop + 32];
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
    }
    uint32_t h[4];
    #pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = half2_bits(v[2 * j] * (1.f / kScale), v[2 * j + 1] * (1.f / kScale));
    __half *C = p.C + (int64_t)bt * p.M * p.ldc;
    if (r0 + lane < p.M) *reinterpret_cast<uint4 *>(C + (int64_t)(r0 + lane) * p.ldc + c0) = make_uint4(h[0], h[1], h[2], h[3]);
    if (mb == nb * BN / kTile) return;
    #pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2 hh = *reinterpret_cast<const __half2 *>(&h[j]);
        stage[warp][(2 * j) * pitch + lane] = __low2half(hh);
        stage[warp][(2 * j + 1) * pitch + lane] = __high2half(hh);
    }
    __syncwarp();
    const int col = lane >> 2, at = (lane & 3) * 8;
    if (c0 + col < p.M && r0 + at < p.M)
        *reinterpret_cast<uint4 *>(C + (int64_t)(c0 + col) * p.ldc + r0 + at) =
            *reinterpret_cast<const uint4 *>(&stage[warp][col * pitch + at]);
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

// Splits of a gram's K: as many as give every pair of CTAs a unit, of at least six stages each, but not
// two, where narrower tiles give as many units without a second launch.  1024 x 4608 in seven splits
// 212 us (all steps), unsplit 248; 1024 x 1024 161 in four, 157 unsplit; 2048 x 2048 259 in two, 249.
int gram_splits(const NewtonShape &s, int *k_per)
{
    const int mb = (s.m + kTile - 1) / kTile, kblk = (s.n + kBK - 1) / kBK;
    const int64_t tiles = (int64_t)s.G * mb * (mb + 1) / 2;
    int want = (int)std::max<int64_t>(1, std::min<int64_t>(num_sms() / 2 / tiles, kblk / 6));
    if (want == 2) want = 1;
    *k_per = (kblk + want - 1) / want;
    return (kblk + *k_per - 1) / *k_per;
}

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
    s->parts = (int)std::min<int64_t>(kNormBlocks, (e + kNormShare - 1) / kNormShare);
    s->x_bytes = up256((size_t)s->G * s->m * s->ldx * 2);
    s->a_bytes = up256((size_t)s->G * s->m * s->lda * 2);
    s->ws = 0;
    if (s->G == 0 || newton_tiny_fits(*s) || newton_small_fits(*s)) return true;
    int k_per;
    const int splits = gram_splits(*s, &k_per), mb = (s->m + kTile - 1) / kTile;
    s->part_bytes = splits > 1 ? (size_t)s->G * mb * (mb + 1) / 2 * splits * kTile * kTile * 4 : 0;
    s->ws = up256((size_t)s->G * s->parts * 4) + 2 * s->x_bytes + 2 * s->a_bytes + s->part_bytes;
    return true;
}

// Columns of a product's tiles: 128 where tiles of 256 would leave half the pairs idle (512 x 512 126 us
// against 154 with 256 always, 1024 x 4608 212 and 232).
int tile_columns(int64_t tiles256) { return tiles256 * 2 <= num_sms() / 2 ? 128 : 256; }

template <int MODE, int BN>
gconv_status launch_tiles(const CUtensorMap &tA, const CUtensorMap &tB, NewtonParams &p, cudaStream_t st)
{
    p.tiles_per = MODE == kApply ? p.n_mblk * ((p.N + BN - 1) / BN) : kTile / BN * p.n_mblk * (p.n_mblk + 1) / 2;
    static bool attr[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GCONV_ERR_CUDA;
    if (!attr[dev]) {
        if (cudaFuncSetAttribute(newton_gemm_kernel<MODE, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) !=
            cudaSuccess)
            return GCONV_ERR_CUDA;
        attr[dev] = true;
    }
    const int64_t units = (int64_t)p.batch * p.tiles_per * p.splits;
    launch_dependent_clusters(newton_gemm_kernel<MODE, BN>, 2 * (unsigned)std::min<int64_t>(units, num_sms() / 2), kThreads, kSmem,
                              2, st, tA, tB, p);
    if (MODE == kGram && p.splits > 1)   // 64 BN / 8 warps a tile
        launch_dependent(newton_sum_kernel<BN>, (unsigned)(p.batch * p.tiles_per * (BN / 8)), 256, 0, st, p);
    return GCONV_OK;
}

template <int MODE>
gconv_status launch_gemm(const CUtensorMap &tA, const CUtensorMap &tB, NewtonParams &p, cudaStream_t st)
{
    p.n_mblk = (p.M + kTile - 1) / kTile;
    p.n_kblk = (p.K + kBK - 1) / kBK;
    if (MODE != kGram) { p.splits = 1; p.k_per = p.n_kblk; }
    const int64_t tiles = (int64_t)p.batch * (MODE == kApply ? p.n_mblk * ((p.N + kTile - 1) / kTile)
                                                             : p.n_mblk * (p.n_mblk + 1) / 2);
    // a gram in splits fills the pairs already
    if (p.splits == 1 && tile_columns(tiles) == 128) return launch_tiles<MODE, 128>(tA, tB, p, st);
    return launch_tiles<MODE, 256>(tA, tB, p, st);
}

gconv_status run_newton(const NewtonShape &s, NewtonIn in, const NewtonOut &out, int steps, const float *coeffs,
                        void *workspace, cudaStream_t st)
{
    unsigned int *err = device_error_word();
    if (!err) return GCONV_ERR_CUDA;
    cudaGetLastError();   // clear a stale error: the check after the launches is about this call
    NewtonOut o = out;
    o.tall = in.tall = s.tall;
    in.rows = s.rows; in.cols = s.cols; in.elems = (int64_t)s.rows * s.cols;
    if (newton_tiny_fits(s)) return newton_tiny_launch(s, in, o, steps, coeffs, st);
    if (newton_small_fits(s)) return newton_small_launch(s, in, o, steps, coeffs, err, st);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    float *part = reinterpret_cast<float *>(ws);
    ws += up256((size_t)s.G * s.parts * 4);
    __half *x[2] = {reinterpret_cast<__half *>(ws), reinterpret_cast<__half *>(ws + s.x_bytes)};
    ws += 2 * s.x_bytes;
    __half *A = reinterpret_cast<__half *>(ws), *P = reinterpret_cast<__half *>(ws + s.a_bytes);
    ws += 2 * s.a_bytes;
    CUtensorMap tX[2], tA, tP;
    if (!half_tmap(&tX[0], x[0], s.n, s.m, s.ldx, s.G) || !half_tmap(&tX[1], x[1], s.n, s.m, s.ldx, s.G) ||
        !half_tmap(&tA, A, s.m, s.m, s.lda, s.G) || !half_tmap(&tP, P, s.m, s.m, s.lda, s.G))
        return GCONV_ERR_CUDA;
    const int64_t share = ((in.elems + s.parts - 1) / s.parts + 7) & ~(int64_t)7;
    const bool v8 = in.elems % 8 == 0;
    const int col_tiles = (s.cols + 31) / 32, row_tiles = (s.rows + 63) / 64;
    for (int g0 = 0; g0 < s.G; g0 += 65535) {   // a grid's y is 16 bits
        const unsigned g = (unsigned)std::min(65535, s.G - g0);
        NewtonIn q = in;
        const int64_t off = (int64_t)g0 * in.elems;
        q.g = static_cast<const uint8_t *>(in.g) + off * (in.g_bf16 ? 2 : 4);
        if (in.m) { q.m = in.m + off; q.m_out = in.m_out + off; }
        float *pg = part + (size_t)g0 * s.parts;
        __half *xg = x[0] + (int64_t)g0 * s.m * s.ldx;
        if (v8) newton_norm_kernel<8><<<dim3(s.parts, g), 256, 0, st>>>(q, pg, share);
        else newton_norm_kernel<1><<<dim3(s.parts, g), 256, 0, st>>>(q, pg, share);
        if (!s.tall && s.n % 8 == 0)
            newton_scale_flat_kernel<<<dim3((unsigned)((in.elems + kNormShare - 1) / kNormShare), g), 256, 0, st>>>(
                q, pg, s.parts, xg);
        else
            newton_scale_kernel<<<dim3((unsigned)(col_tiles * row_tiles), g), 256, 0, st>>>(q, pg, s.parts, xg, s.ldx,
                                                                                            col_tiles);
    }
    NewtonParams p{};
    p.batch = s.G; p.err = err; p.wait_ns = (uint64_t)wait_limit();
    p.part = reinterpret_cast<float *>(ws);
    p.M = s.m;
    p.o = o;
    for (int k = 0; k < steps; ++k) {
        const float *c = coeffs ? coeffs + 3 * k : kNewtonCoeffs;
        p.N = s.m; p.K = s.n; p.ldc = s.lda; p.C = A;
        p.splits = gram_splits(s, &p.k_per);
        gconv_status r = launch_gemm<kGram>(tX[k & 1], tX[k & 1], p, st);
        if (r != GCONV_OK) return r;
        p.K = s.m; p.C = P; p.A = A;
        p.a = c[0]; p.b = c[1]; p.c = c[2];
        r = launch_gemm<kPoly>(tA, tA, p, st);
        if (r != GCONV_OK) return r;
        p.N = s.n; p.ldc = s.ldx; p.C = x[(k + 1) & 1];
        p.last = k + 1 == steps;
        r = launch_gemm<kApply>(tP, tX[k & 1], p, st);
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
    return newton_shape(matrices, &s) ? s.ws : (size_t)-1;
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
    if (s.ws && (!workspace || workspace_bytes < s.ws)) return GCONV_ERR_WORKSPACE;
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
    if (s.ws && (!workspace || workspace_bytes < s.ws)) return GCONV_ERR_WORKSPACE;
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
