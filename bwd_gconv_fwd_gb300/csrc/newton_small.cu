// newton_small.cu -- all Newton-Schulz steps of a matrix whose shorter side is at most 128
// in one launch: a cluster of thread blocks a matrix, each holding a slice of X's columns in
// shared memory from the first step to the last.
//
// A step of block r with its slice X_r (m x ns):
//   S_r = X_r X_r^T                    tcgen05, 128 x 128 accumulator in tensor memory
//   A   = sum over r of S_r            rows dealt over the blocks, read through distributed
//                                      shared memory in rank order, A sent to every block
//   P   = a I + b A + c A A            every block for itself
//   X_r = P X_r                        in place
// What a step costs is its chain of waits (three products, two cluster barriers), not its
// bytes or operations, which is why a matrix stays on one cluster.
//
// The 128-byte swizzled tile of 64 columns x 128 rows that the first product reads with rows
// as its outer side (K-major) is, with the roles of rows and columns exchanged, the tile
// that the last product reads with rows as its inner side (N-major): one copy of X serves both.
#include "newton.cuh"

#include <algorithm>
#include <type_traits>

namespace gconv {

namespace {

constexpr int kSmallThreads = 512, kSmallWarps = 16;
constexpr uint32_t kChunkBytes = 16384;       // 64 columns x 128 rows of fp16
constexpr int kMaxChunks = 8;                 // a slice of 512 columns: all of tensor memory
constexpr uint64_t kSmallDrainNs = 1000000000ull;

struct SmallParams {
    NewtonIn in;
    NewtonOut out;
    int m, n, steps, slice;                   // slice: columns a block holds, a multiple of 64
    int cluster;
    unsigned int *err;
    uint64_t wait_ns;
    float coeffs[3 * kNewtonSteps];
};

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_cluster2(uint32_t addr, uint32_t a, uint32_t b)
{
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

__device__ __forceinline__ void st_cluster_f(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Shared-memory writes of the threads behind the next barrier before tensor-core reads after it:
// within the block, and into the others of the cluster.  (The fence over all memory takes some
// hundred cycles more, three times a step.)
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.proxy.async.shared::cluster;" ::: "memory"); }

// Byte offset of the 16-byte piece that holds column `col` of row `row`: 64-column chunks of
// 128-byte rows, pieces exchanged by the row's last three bits (the 128-byte swizzle).
__device__ __forceinline__ uint32_t piece(int row, int col)
{
    return (uint32_t)(col >> 6) * kChunkBytes + (uint32_t)row * 128u + (uint32_t)((((col & 63) >> 3) ^ (row & 7)) << 4);
}

// V elements of the matrix to orthogonalise, at element i of the caller's tensors.  FIRST:
// the sweep that also writes the updated momentum.
template <int V, bool FIRST>
__device__ __forceinline__ void read_u(const NewtonIn &p, int64_t i, float (&u)[V])
{
    if constexpr (V == 4) {
        if (p.g_bf16) {
            const uint2 raw = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p.g) + i);
            const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162 *>(&raw.x);
            const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162 *>(&raw.y);
            u[0] = __low2float(a); u[1] = __high2float(a); u[2] = __low2float(b); u[3] = __high2float(b);
        } else {
            const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.g) + i);
            u[0] = v.x; u[1] = v.y; u[2] = v.z; u[3] = v.w;
        }
    } else {
        u[0] = load_g(p, i);
    }
    if (!p.m) return;
    float m[V];
    const float *src = FIRST ? p.m : p.m_out;
    if constexpr (V == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(src + i);
        m[0] = v.x; m[1] = v.y; m[2] = v.z; m[3] = v.w;
    } else {
        m[0] = src[i];
    }
    if (FIRST) {
        #pragma unroll
        for (int k = 0; k < V; ++k) m[k] = fmaf(p.beta, m[k], u[k]);
        if constexpr (V == 4) *reinterpret_cast<float4 *>(p.m_out + i) = make_float4(m[0], m[1], m[2], m[3]);
        else p.m_out[i] = m[0];
    }
    #pragma unroll
    for (int k = 0; k < V; ++k) u[k] = lookahead(p, u[k], m[k]);
}

// grid: G clusters of p.cluster blocks.
template <int V>
__global__ void __launch_bounds__(kSmallThreads, 1) newton_small_kernel(const __grid_constant__ SmallParams p)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar, bar_drain;
    __shared__ uint32_t tmem_sh;
    __shared__ float warp_sum[kSmallWarps], rank_sum[16];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t CS = (uint32_t)p.cluster, rank = cluster_rank();
    const int mat = blockIdx.x / p.cluster;
    const int c0 = (int)rank * p.slice;
    const int width = min(p.slice, max(0, p.n - c0));       // columns of X here
    const int chunks = p.slice >> 6;
    const int live = (width + 63) >> 6;                     // chunks that hold columns
    const uint32_t sbase = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *sgen = smem_raw + (sbase - ptx::smem_u32(smem_raw));
    const uint32_t oX = 0, oA = (uint32_t)chunks * kChunkBytes, oP = oA + 2 * kChunkBytes;   // P, or the 64 KB of sums
    const int m16 = (p.m + 15) & ~15;

    if (tid == 0) {
        ptx::mbar_init(ptx::smem_u32(&bar), 1);
        ptx::mbar_init(ptx::smem_u32(&bar_drain), 1);
        ptx::fence_mbar_init();
    }
    if (warp == 0) {
        ptx::tmem_alloc(ptx::smem_u32(&tmem_sh), 512);
        ptx::tmem_relinquish();
    }
    for (uint32_t i = tid * 16; i < (uint32_t)chunks * kChunkBytes; i += kSmallThreads * 16)
        *reinterpret_cast<uint4 *>(sgen + oX + i) = make_uint4(0, 0, 0, 0);

    // The slice as it lies in memory: rows of `wide` consecutive elements, `rows` of them
    // `pitch` apart.  LPR lanes take a row, V elements a lane.
    const int rows = p.in.tall ? width : p.m, wide = p.in.tall ? p.m : width;
    const int pitch = p.in.cols;
    const int64_t base = (int64_t)mat * p.in.elems + (p.in.tall ? (int64_t)c0 * pitch : c0);
    int lpr = 1;
    while (lpr < 32 && lpr * V < wide) lpr <<= 1;
    const int rstep = kSmallThreads / lpr, cstep = lpr * V;
    const int r_first = tid / lpr, c_first = (tid % lpr) * V;

    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    constexpr int kBatch = V == 4 ? 4 : 8;                  // reads in flight
    auto sweep = [&](auto first, auto use) {
        int r = r_first, c = c_first;
        while (r < rows) {
            float u[kBatch][V];
            int rr[kBatch], cc[kBatch];
            #pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                rr[k] = r; cc[k] = c;
                if (r < rows && c < wide) read_u<V, decltype(first)::value>(p.in, base + (int64_t)r * pitch + c, u[k]);
                c += cstep;
                if (c >= wide) { c = c_first; r += rstep; }
            }
            #pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (rr[k] < rows && cc[k] < wide) use(rr[k], cc[k], u[k]);
        }
    };

    float s = 0.f;
    sweep(std::true_type{}, [&](int, int, const float (&u)[V]) {
        #pragma unroll
        for (int k = 0; k < V; ++k) s = fmaf(u[k], u[k], s);
    });
    #pragma unroll
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (lane == 0) warp_sum[warp] = s;
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_sh;
    cluster_sync();   // the others' shared memory may be written from here on
    if (tid < (int)CS) {
        float t = 0.f;
        for (int k = 0; k < kSmallWarps; ++k) t += warp_sum[k];
        st_cluster_f(map_to(ptx::smem_u32(&rank_sum[rank]), (uint32_t)tid), t);
    }
    cluster_sync();
    float total = 0.f;
    for (uint32_t k = 0; k < CS; ++k) total += rank_sum[k];
    const float inv = kNewtonScale / (sqrtf(total) + p.in.eps);
    sweep(std::false_type{}, [&](int r, int c, const float (&u)[V]) {
        if (p.in.tall) {
            #pragma unroll
            for (int k = 0; k < V; ++k)
                *reinterpret_cast<__half *>(sgen + oX + piece(c + k, r) + (r & 7) * 2) = __float2half_rn(u[k] * inv);
        } else if constexpr (V == 4) {
            *reinterpret_cast<uint2 *>(sgen + oX + piece(r, c) + (c & 7) * 2) =
                make_uint2(half2_bits(u[0] * inv, u[1] * inv), half2_bits(u[2] * inv, u[3] * inv));
        } else {
            *reinterpret_cast<__half *>(sgen + oX + piece(r, c) + (c & 7) * 2) = __float2half_rn(u[0] * inv);
        }
    });
    ptx::fence_proxy_async_smem();
    __syncthreads();

    uint32_t phase = 0;
    bool ok = true;
    // waits for the products committed last; after a wait that gave up, none waits again
    auto products_done = [&] {
        if (ok && !ptx::mbar_wait(ptx::smem_u32(&bar), phase, p.wait_ns)) {
            ok = false;
            if (lane == 0) raise_device_error(p.err, DEVERR_WAIT_TIMEOUT);
        }
        phase ^= 1u;
        ptx::tc_fence_after();
        __syncwarp();
    };
    const int q = warp & 3, cb = warp >> 2;                 // TMEM lane quarter, 32-column block
    const int row = q * 32 + lane;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;

    for (int step = 0; step < p.steps; ++step) {
        const float a = p.coeffs[3 * step], b = p.coeffs[3 * step + 1], c = p.coeffs[3 * step + 2];
        // ---- S = X X^T ----
        if (tid == 0) {
            const uint32_t idesc = idesc_f16(128, m16, 0);
            uint32_t acc = 0;
            for (int k = 0; k < max(live, 1); ++k)
                #pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint64_t d = ptx::smem_desc(sbase + oX + k * kChunkBytes + j * 32, 16, 1024, 2);
                    ptx::mma_f16(tmem, d, d, idesc, acc);
                    acc = 1;
                }
            ptx::mma_commit(ptx::smem_u32(&bar));
        }
        products_done();
        if (cb * 32 < m16) {
            uint32_t v[2][16];
            ptx::tmem_ld16(tmem + lanes + cb * 32, v[0]);
            ptx::tmem_ld16(tmem + lanes + cb * 32 + 16, v[1]);
            ptx::tmem_ld_wait();
            const float *f = reinterpret_cast<const float *>(&v[0][0]);
            if (CS == 1) {
                #pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint4 h;
                    h.x = half2_bits(f[8 * j] * (1.f / kNewtonScale), f[8 * j + 1] * (1.f / kNewtonScale));
                    h.y = half2_bits(f[8 * j + 2] * (1.f / kNewtonScale), f[8 * j + 3] * (1.f / kNewtonScale));
                    h.z = half2_bits(f[8 * j + 4] * (1.f / kNewtonScale), f[8 * j + 5] * (1.f / kNewtonScale));
                    h.w = half2_bits(f[8 * j + 6] * (1.f / kNewtonScale), f[8 * j + 7] * (1.f / kNewtonScale));
                    *reinterpret_cast<uint4 *>(sgen + oA + piece(row, cb * 32 + 8 * j)) = h;
                }
            } else {
                // 512-byte rows of fp32, 16-byte pieces exchanged by the row's last three bits
                #pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<float4 *>(sgen + oP + row * 512 + (((cb * 8 + j) ^ (row & 7)) << 4)) =
                        make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
            }
        }
        if (CS > 1) {
            cluster_sync();
            // This block adds rows rank, rank + CS, ... of the m16 (rows m to m16 are sums of zeros).
            // It begins with its own part and goes round the others, so that at any time the
            // blocks read from, and write to, different ones.
            const int pieces = m16 / 4, mine = (m16 - (int)rank + (int)CS - 1) / (int)CS;
            for (int i = tid; i < mine * pieces; i += kSmallThreads) {
                const int k_row = i / pieces, pc = i - k_row * pieces, r = (int)rank + k_row * (int)CS;
                const uint32_t at = sbase + oP + r * 512 + ((pc ^ (r & 7)) << 4);
                float4 part[8];
                #pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < (int)CS) part[k] = ld_cluster4(map_to(at, (rank + k) & (CS - 1)));
                float4 t = part[0];
                #pragma unroll
                for (int k = 1; k < 8; ++k)
                    if (k < (int)CS) { t.x += part[k].x; t.y += part[k].y; t.z += part[k].z; t.w += part[k].w; }
                const uint32_t lo = half2_bits(t.x * (1.f / kNewtonScale), t.y * (1.f / kNewtonScale));
                const uint32_t hi = half2_bits(t.z * (1.f / kNewtonScale), t.w * (1.f / kNewtonScale));
                const uint32_t to = sbase + oA + piece(r, pc * 4) + ((pc & 1) << 3);
                #pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < (int)CS) st_cluster2(map_to(to, (rank + k) & (CS - 1)), lo, hi);
            }
            fence_cluster();
            cluster_sync();
        } else {
            ptx::fence_proxy_async_smem();
            ptx::tc_fence_before();
            __syncthreads();
        }
        // ---- P = a I + b A + c A A ----
        if (tid == 0) {
            if (CS > 1) fence_cluster();   // the others' writes
            ptx::tc_fence_after();
            const uint32_t idesc = idesc_f16(128, m16, 0);
            for (int k = 0; k < m16 / 16; ++k) {
                const uint64_t d = ptx::smem_desc(sbase + oA + (k >> 2) * kChunkBytes + (k & 3) * 32, 16, 1024, 2);
                ptx::mma_f16(tmem + 128, d, d, idesc, k > 0);
            }
            ptx::mma_commit(ptx::smem_u32(&bar));
        }
        products_done();
        if (cb * 32 < m16) {
            uint32_t v[2][16];
            ptx::tmem_ld16(tmem + lanes + 128 + cb * 32, v[0]);
            ptx::tmem_ld16(tmem + lanes + 128 + cb * 32 + 16, v[1]);
            ptx::tmem_ld_wait();
            const float *f = reinterpret_cast<const float *>(&v[0][0]);
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t at = piece(row, cb * 32 + 8 * j);
                const uint4 lin = *reinterpret_cast<const uint4 *>(sgen + oA + at);
                const uint32_t w[4] = {lin.x, lin.y, lin.z, lin.w};
                uint32_t h[4];
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 l = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
                    const int col = cb * 32 + 8 * j + 2 * k;
                    float x = fmaf(c * (1.f / kNewtonScale), f[8 * j + 2 * k], b * l.x);
                    float y = fmaf(c * (1.f / kNewtonScale), f[8 * j + 2 * k + 1], b * l.y);
                    if (col == row) x += a * kNewtonScale;
                    if (col + 1 == row) y += a * kNewtonScale;
                    h[k] = half2_bits(x, y);
                }
                *reinterpret_cast<uint4 *>(sgen + oP + at) = make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncthreads();
        // ---- X = P X ----
        if (tid == 0) {
            ptx::tc_fence_after();
            for (int g = 0; g < max(live, 1); g += 4) {
                const int n = min(4, max(live, 1) - g) * 64;
                const uint32_t idesc = idesc_f16(128, n, 1);
                for (int k = 0; k < m16 / 16; ++k)
                    ptx::mma_f16(tmem + g * 64,
                                 ptx::smem_desc(sbase + oP + (k >> 2) * kChunkBytes + (k & 3) * 32, 16, 1024, 2),
                                 ptx::smem_desc(sbase + oX + g * kChunkBytes + k * 2048, kChunkBytes, 1024, 2), idesc, k > 0);
            }
            ptx::mma_commit(ptx::smem_u32(&bar));
        }
        products_done();
        if (step + 1 < p.steps) {
            for (int blk = cb; blk < live * 2; blk += 4) {
                uint32_t v[2][16];
                ptx::tmem_ld16(tmem + lanes + blk * 32, v[0]);
                ptx::tmem_ld16(tmem + lanes + blk * 32 + 16, v[1]);
                ptx::tmem_ld_wait();
                const float *f = reinterpret_cast<const float *>(&v[0][0]);
                if (row < p.m) {
                    #pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint4 h;
                        h.x = half2_bits(f[8 * j] * (1.f / kNewtonScale), f[8 * j + 1] * (1.f / kNewtonScale));
                        h.y = half2_bits(f[8 * j + 2] * (1.f / kNewtonScale), f[8 * j + 3] * (1.f / kNewtonScale));
                        h.z = half2_bits(f[8 * j + 4] * (1.f / kNewtonScale), f[8 * j + 5] * (1.f / kNewtonScale));
                        h.w = half2_bits(f[8 * j + 6] * (1.f / kNewtonScale), f[8 * j + 7] * (1.f / kNewtonScale));
                        *reinterpret_cast<uint4 *>(sgen + oX + piece(row, blk * 32 + 8 * j)) = h;
                    }
                }
            }
            ptx::fence_proxy_async_smem();
            ptx::tc_fence_before();
            __syncthreads();
            if (tid == 0) ptx::tc_fence_after();
        }
    }

    // ---- the result, through shared memory where a warp's lanes hold a column ----
    const float back = 1.f / (kNewtonScale * kNewtonScale);
    const int64_t out0 = (int64_t)mat * p.m * p.n;
    __syncthreads();   // every warp past its last wait: X, A and P are free
    float *stage = reinterpret_cast<float *>(sgen) + warp * 32 * 33;
    for (int blk = cb; blk < live * 2; blk += 4) {
        uint32_t v[2][16];
        ptx::tmem_ld16(tmem + lanes + blk * 32, v[0]);
        ptx::tmem_ld16(tmem + lanes + blk * 32 + 16, v[1]);
        ptx::tmem_ld_wait();
        const float *f = reinterpret_cast<const float *>(&v[0][0]);
        if (p.out.tall) {
            #pragma unroll
            for (int j = 0; j < 32; ++j) {
                const int col = blk * 32 + j;
                if (row < p.m && col < width) store_result(p.out, out0 + (int64_t)(c0 + col) * p.m + row, f[j] * back);
            }
        } else {
            #pragma unroll
            for (int j = 0; j < 32; ++j) stage[lane * 33 + j] = f[j] * back;
            __syncwarp();
            store_rows(p.out, out0 + (int64_t)(q * 32) * p.n + c0 + blk * 32, p.n, min(32, p.m - q * 32),
                       min(32, width - blk * 32), stage, lane);
            __syncwarp();
        }
    }
    // every product has ended before tensor memory is released
    if (tid == 0) {
        ptx::mma_commit(ptx::smem_u32(&bar_drain));
        if (!ptx::mbar_wait(ptx::smem_u32(&bar_drain), 0, kSmallDrainNs)) raise_device_error(p.err, DEVERR_WAIT_TIMEOUT);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 0) ptx::tmem_dealloc(tmem, 512);
}

// Blocks a matrix: as few as keep a slice at kMaxChunks, more while they are idle and slices
// are longer than two chunks.
int small_cluster(const NewtonShape &s, int *slice)
{
    for (int cs = 1; cs <= 8; cs *= 2) {
        const int sl = ((s.n + cs - 1) / cs + 63) / 64 * 64;
        if (sl > kMaxChunks * 64) continue;
        if (cs < 8 && sl > 128 && (int64_t)s.G * cs * 2 <= num_sms()) continue;
        *slice = sl;
        return cs;
    }
    return 0;
}

}  // namespace

bool newton_small_fits(const NewtonShape &s)
{
    int slice;
    return s.m <= 128 && small_cluster(s, &slice) > 0 && (int64_t)s.G * 8 < INT32_MAX;
}

gconv_status newton_small_launch(const NewtonShape &s, const NewtonIn &in, const NewtonOut &out, int steps,
                                 const float *coeffs, unsigned int *err, cudaStream_t st)
{
    SmallParams p{};
    p.in = in; p.out = out; p.m = s.m; p.n = s.n; p.steps = steps;
    p.cluster = small_cluster(s, &p.slice);
    p.err = err; p.wait_ns = (uint64_t)wait_limit();
    for (int k = 0; k < 3 * steps; ++k) p.coeffs[k] = coeffs ? coeffs[k] : kNewtonCoeffs[k % 3];
    // X, A, then P or (several blocks) 64 KB of partial sums; the result is staged over them.
    // More than half an SM's shared memory: two blocks on one SM would wait for each other's
    // tensor memory, and two clusters that each hold what the other waits for would never end.
    const size_t smem = std::max<size_t>(1024 + (size_t)(p.slice / 64 + 2 + (p.cluster > 1 ? 4 : 2)) * kChunkBytes, 120 * 1024);
    const bool vec = s.cols % 4 == 0;
    static bool attr[64][2] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GCONV_ERR_CUDA;
    auto fn = vec ? newton_small_kernel<4> : newton_small_kernel<1>;
    if (!attr[dev][vec]) {
        const int most = 1024 + (kMaxChunks + 6) * (int)kChunkBytes;
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) return GCONV_ERR_CUDA;
        attr[dev][vec] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(s.G * p.cluster));
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)p.cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, fn, p);
    return cudaGetLastError() == cudaSuccess ? GCONV_OK : GCONV_ERR_CUDA;
}

}  // namespace gconv
