// newton_small.cu -- all Newton-Schulz steps of a matrix whose shorter side is at most 128
// in one launch: a cluster of thread blocks a matrix, each holding a slice of X's columns in
// shared memory from the first step to the last.
//
// A step of block r with its slice X_r (m x ns):
//   S_r = X_r X_r^T                    tcgen05, 128 x 128 accumulator in tensor memory
//   A   = sum over r of S_r            each block sends every other its share of S_r's rows, adds the
//                                      shares it gets in rank order, and sends its rows of A back
//   P   = a I + b A + c A A            every block for itself
//   X_r = P X_r                        in place
// What a step costs is its chain of waits (three products, two exchanges), not its bytes or
// operations, which is why a matrix stays on one cluster.  The exchanges are bulk copies between
// the blocks' shared memory that signal the receiver's barrier: reading the others' memory between
// two cluster barriers cost half of a step (128 x 1200: 7500 of 14700 cycles).
//   Measured, five steps: 64 x 576 24 us, two of 128 x 1200 45, 128 x 4096 53, 64 x 256 23; one launch a
// product (newton.cu) takes 81, 103, 113 and 64.  A step is 4 to 9 us of latency: the two products' fill
// and drain, two exchanges and three turns between the kinds of accesses to shared memory.
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
constexpr int kMaxCluster = 16;
constexpr int kSmallPitch = 36;               // floats of a staged row of the result
constexpr size_t kSmallSmem = 1024 + 14 * (size_t)kChunkBytes;
constexpr uint64_t kSmallDrainNs = 1000000000ull;

struct SmallParams {
    NewtonIn in;
    NewtonOut out;
    int m, n, steps, slice;                   // slice: columns a block holds, a multiple of 64
    int cluster;
    int m16, pitch, keep, ordered;            // m up to 16; bytes of a row of S_r, a power of two; see sweep
    uint32_t oA, oS, oR, oOut;                // A; S_r, and P in its place; the shares received; the result's stage
    unsigned int *err;
    uint64_t wait_ns;
    float coeffs[3 * kNewtonSteps];
};

__device__ __forceinline__ void st_cluster_f(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// `bytes` (a multiple of 16) of this block's shared memory to the same or another offset of block
// `rank`'s, counted on its barrier `bar` (an offset like the others).
__device__ __forceinline__ void send(uint32_t to, uint32_t from, uint32_t bytes, uint32_t bar, uint32_t rank)
{
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(ptx::map_to(to, rank)), "r"(from), "r"(bytes), "r"(ptx::map_to(bar, rank)) : "memory");
}

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

// V elements of what a call writes.
template <int V>
__device__ __forceinline__ void put_results(const NewtonOut &o, int64_t at, const float (&v)[V])
{
    if constexpr (V == 4) {
        __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
        const float4 f = make_float4(v[0], v[1], v[2], v[3]);
        if (o.muon) {
            *reinterpret_cast<float4 *>(o.w_out + at) = f;
            if (o.w_bf16) *reinterpret_cast<uint2 *>(o.w_bf16 + at) = *reinterpret_cast<uint2 *>(h);
        } else if (o.out_bf16) {
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(o.out) + at) = *reinterpret_cast<uint2 *>(h);
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(o.out) + at) = f;
        }
    } else {
        put_result(o, at, v[0]);
    }
}

// A staged 32 x 32 block of the result to rows n elements apart from element `at`; `rows` and `cols`
// of it exist.  32 / V lanes a row; the weights are read for the whole block before any is written.
template <int V>
__device__ __forceinline__ void store_block(const NewtonOut &o, int64_t at, int n, int rows, int cols, const float *stage, int lane)
{
    constexpr int per = V, rounds = 32 / per;               // rows a store, stores
    const int r0 = lane / (32 / V), c = lane % (32 / V) * V;
    if (c >= cols) return;
    float w[rounds][V];
    if (o.muon) {
        #pragma unroll
        for (int k = 0; k < rounds; ++k)
            if (k * per + r0 < rows) {
                const Pack<float, V> p = *reinterpret_cast<const Pack<float, V> *>(o.w + at + (int64_t)(k * per + r0) * n + c);
                #pragma unroll
                for (int e = 0; e < V; ++e) w[k][e] = p.v[e];
            }
    }
    #pragma unroll
    for (int k = 0; k < rounds; ++k) {
        const int r = k * per + r0;
        if (r >= rows) continue;
        const Pack<float, V> p = *reinterpret_cast<const Pack<float, V> *>(stage + r * kSmallPitch + c);
        float v[V];
        #pragma unroll
        for (int e = 0; e < V; ++e) v[e] = o.muon ? fmaf(-o.rate, p.v[e], o.keep * w[k][e]) : p.v[e];
        put_results<V>(o, at + (int64_t)r * n + c, v);
    }
}

// grid: G clusters of p.cluster blocks.
template <int V>
__global__ void __launch_bounds__(kSmallThreads, 1) newton_small_kernel(const __grid_constant__ SmallParams p)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar, bar_drain, bar_shares, bar_rows;
    __shared__ uint32_t tmem_sh;
    __shared__ float warp_sum[kSmallWarps], rank_sum[kMaxCluster];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t CS = (uint32_t)p.cluster, rank = ptx::cluster_rank();
    const int mat = blockIdx.x / p.cluster;
    const int c0 = (int)rank * p.slice;
    const int width = min(p.slice, max(0, p.n - c0));       // columns of X here
    const int chunks = p.slice >> 6;
    const int live = (width + 63) >> 6;                     // chunks that hold columns
    const uint32_t sbase = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *sgen = smem_raw + (sbase - ptx::smem_u32(smem_raw));
    const uint32_t oX = 0, oA = p.oA, oP = p.oS;
    const int m16 = p.m16;

    if (tid == 0) {
        ptx::mbar_init(ptx::smem_u32(&bar), 1);
        ptx::mbar_init(ptx::smem_u32(&bar_drain), 1);
        ptx::mbar_init(ptx::smem_u32(&bar_shares), 1);
        ptx::mbar_init(ptx::smem_u32(&bar_rows), 1);
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
    // The first sweep adds the squares, the second scales; between them the values wait in what
    // A, S and the shares will use, where that is large enough, else they are read again.  Where they reach
    // the shares (`ordered`), no block may send one before every block of the cluster has ended its
    // second sweep: a block with few columns, or none, would be there long before the others.  (A Muon step of
    // 256 x 64, whose values do not reach, 30.8 us without the barrier and 31.4 with it.)
    constexpr int kBatch = 8;                               // reads in flight
    float *kept = reinterpret_cast<float *>(sgen + p.oA) + tid * V;
    auto sweep = [&](auto first, auto use) {
        int r = r_first, c = c_first, n = 0;
        while (r < rows) {
            float u[kBatch][V];
            int rr[kBatch], cc[kBatch];
            #pragma unroll
            for (int k = 0; k < kBatch; ++k, ++n) {
                rr[k] = r; cc[k] = c;
                if (r < rows && c < wide) {
                    if (!decltype(first)::value && p.keep) {
                        const Pack<float, V> v = *reinterpret_cast<const Pack<float, V> *>(kept + n * kSmallThreads * V);
                        #pragma unroll
                        for (int e = 0; e < V; ++e) u[k][e] = v.v[e];
                    } else {
                        read_u<V, decltype(first)::value>(p.in, base + (int64_t)r * pitch + c, u[k]);
                    }
                }
                c += cstep;
                if (c >= wide) { c = c_first; r += rstep; }
            }
            #pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (rr[k] < rows && cc[k] < wide) use(rr[k], cc[k], n - kBatch + k, u[k]);
        }
    };

    float s = 0.f;
    sweep(std::true_type{}, [&](int, int, int n, const float (&u)[V]) {
        Pack<float, V> v;
        #pragma unroll
        for (int k = 0; k < V; ++k) { s = fmaf(u[k], u[k], s); v.v[k] = u[k]; }
        if (p.keep) *reinterpret_cast<Pack<float, V> *>(kept + n * kSmallThreads * V) = v;
    });
    #pragma unroll
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (lane == 0) warp_sum[warp] = s;
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_sh;
    ptx::cluster_sync();   // the others' shared memory may be written from here on
    if (tid < (int)CS) {
        float t = 0.f;
        for (int k = 0; k < kSmallWarps; ++k) t += warp_sum[k];
        st_cluster_f(ptx::map_to(ptx::smem_u32(&rank_sum[rank]), (uint32_t)tid), t);
    }
    ptx::cluster_sync();
    float total = 0.f;
    for (uint32_t k = 0; k < CS; ++k) total += rank_sum[k];
    const float inv = unit_factor(kNewtonScale, total, p.in.eps);
    sweep(std::false_type{}, [&](int r, int c, int, const float (&u)[V]) {
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
    if (p.ordered) ptx::cluster_arrive();   // this block's values have been read; waited for before the first share is sent

    uint32_t phase = 0;
    bool ok = true;
    // Waits, every thread, for a barrier's phase; after a wait that gave up, none waits again.
    auto wait_for = [&](uint64_t *b, uint32_t parity) {
        if (ok && !ptx::mbar_wait(ptx::smem_u32(b), parity, p.wait_ns)) {
            ok = false;
            if (lane == 0) raise_device_error(p.err, DEVERR_WAIT_TIMEOUT);
        }
    };
    auto products_done = [&] {
        wait_for(&bar, phase);
        phase ^= 1u;
        ptx::tc_fence_after();
        __syncwarp();
    };
    const int share = m16 / (int)CS;                        // rows of A this block adds up, from share * rank
    const uint32_t share_bytes = (uint32_t)share * (uint32_t)p.pitch;
    const int swap = (p.pitch >> 4) < 8 ? (p.pitch >> 4) - 1 : 7;   // which pieces of a row of S change places
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
                // rows of fp32, 16-byte pieces exchanged by the row's last bits
                #pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (row < m16 && cb * 32 + 4 * j < m16)
                        *reinterpret_cast<float4 *>(sgen + p.oS + row * p.pitch + (((cb * 8 + j) ^ (row & swap)) << 4)) =
                            make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
            }
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncthreads();
        if (step == 0 && p.ordered) ptx::cluster_wait();
        if (CS > 1) {
            // What a block overwrites here has been read: in the first step by the barrier above (rows of A come
            // only after this block's share, which it sends behind its second sweep); later, S was received
            // everywhere before A's rows came back last step, R was added up before its rows of A left,
            // and A's old rows were read before the sums that replace them were sent.
            const uint32_t bar_s = ptx::smem_u32(&bar_shares), bar_r = ptx::smem_u32(&bar_rows);
            const int a_chunks = (m16 + 63) >> 6;
            if (tid == 0 && ok) {   // not at a barrier whose last phase may still be open
                ptx::mbar_arrive_expect_tx(bar_s, CS * share_bytes);
                ptx::mbar_arrive_expect_tx(bar_r, (CS - 1) * (uint32_t)(a_chunks * share * 128));
            }
            if (tid < (int)CS && ok)
                send(sbase + p.oR + rank * share_bytes, sbase + p.oS + (uint32_t)tid * share_bytes, share_bytes, bar_s,
                     (uint32_t)tid);
            wait_for(&bar_shares, step & 1);
            const int pieces = m16 / 4;
            for (int i = tid; i < share * pieces; i += kSmallThreads) {
                const int k_row = i / pieces, pc = i - k_row * pieces, r = (int)rank * share + k_row;
                const uint8_t *from = sgen + p.oR + k_row * p.pitch + ((pc ^ (r & swap)) << 4);
                float4 t = *reinterpret_cast<const float4 *>(from);
                #pragma unroll 8
                for (uint32_t k = 1; k < CS; ++k) {
                    const float4 u = *reinterpret_cast<const float4 *>(from + k * share_bytes);
                    t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
                }
                *reinterpret_cast<uint2 *>(sgen + oA + piece(r, pc * 4) + ((pc & 1) << 3)) =
                    make_uint2(half2_bits(t.x * (1.f / kNewtonScale), t.y * (1.f / kNewtonScale)),
                               half2_bits(t.z * (1.f / kNewtonScale), t.w * (1.f / kNewtonScale)));
            }
            ptx::fence_proxy_async_smem();
            __syncthreads();
            if (tid < (int)CS * a_chunks && ok) {
                const uint32_t to = (uint32_t)tid % CS, at = sbase + oA + (uint32_t)tid / CS * kChunkBytes + rank * (uint32_t)share * 128u;
                if (to != rank) send(at, at, (uint32_t)share * 128u, bar_r, to);
            }
            wait_for(&bar_rows, step & 1);
        }
        // ---- P = a I + b A + c A A ----
        if (tid == 0) {
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
    __syncthreads();   // every warp past its last wait: X and P are free
    float *stage = reinterpret_cast<float *>(sgen + p.oOut) + warp * 32 * kSmallPitch;
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
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<float4 *>(stage + lane * kSmallPitch + 4 * j) =
                    make_float4(f[4 * j] * back, f[4 * j + 1] * back, f[4 * j + 2] * back, f[4 * j + 3] * back);
            __syncwarp();
            store_block<V>(p.out, out0 + (int64_t)(q * 32) * p.n + c0 + blk * 32, p.n, p.m - q * 32, width - blk * 32, stage, lane);
            __syncwarp();
        }
    }
    // every product has ended before tensor memory is released
    if (tid == 0) {
        ptx::mma_commit(ptx::smem_u32(&bar_drain));
        if (!ptx::mbar_wait(ptx::smem_u32(&bar_drain), 0, kSmallDrainNs)) raise_device_error(p.err, DEVERR_WAIT_TIMEOUT);
    }
    // Copies to and from this block have ended: each was waited for where it arrived, or, after a wait
    // that gave up, has the time to land.
    if (__syncthreads_or(!ok) && tid == 0) ptx::let_pass(kSmallDrainNs);
    __syncwarp();
    ptx::tc_fence_before();
    ptx::cluster_sync();
    if (warp == 0) ptx::tmem_dealloc(tmem, 512);
}

// Where a block keeps what (the kernel's oA, oS, oR), and the bytes in all.
size_t small_layout(const NewtonShape &s, int cluster, int slice, SmallParams *p)
{
    const int m16 = (s.m + 15) & ~15, a_chunks = (m16 + 63) / 64;
    int pitch = 64;
    while (pitch < m16 * 4) pitch <<= 1;
    p->m16 = m16;
    p->pitch = pitch;
    p->oA = (uint32_t)(slice / 64) * kChunkBytes;
    p->oS = p->oA + a_chunks * kChunkBytes;
    const uint32_t sums = cluster > 1 ? (uint32_t)(m16 * pitch) : 0;
    p->oR = p->oS + std::max<uint32_t>(sums, a_chunks * kChunkBytes);
    // the result is staged where nothing is read or sent any more: not over A
    constexpr uint32_t stage = kSmallWarps * 32 * kSmallPitch * 4;
    p->oOut = p->oA >= stage ? 0 : p->oS;
    return 1024 + std::max(p->oR + sums, p->oOut + stage);
}

// Whether a cluster of sixteen blocks of this kernel fits the current device.
bool sixteen_fit()
{
    static int cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return false;
    }
    if (!cache[dev]) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kMaxCluster);
        cfg.blockDim = dim3(kSmallThreads);
        cfg.dynamicSmemBytes = kSmallSmem;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = kMaxCluster;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        auto fn = newton_small_kernel<4>;
        const bool ok = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmallSmem) == cudaSuccess &&
                        cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                        cudaOccupancyMaxActiveClusters(&n, fn, &cfg) == cudaSuccess && n > 0;
        cudaGetLastError();
        cache[dev] = ok ? 1 : -1;
    }
    return cache[dev] > 0;
}

// Blocks a matrix: as few as their shared memory allows, more while most SMs are idle and a slice is
// longer than one chunk (64 x 576: two blocks 32 us, four 26, eight 24; 16 of them, which as clusters of
// eight do not all run at once, 26 in fours and 47 in eights).  Clusters of sixteen, which not every
// part of the device can hold, only where eight do not fit.
int small_cluster(const NewtonShape &s, int *slice)
{
    for (int cs = 1; cs <= kMaxCluster; cs *= 2) {
        const int sl = ((s.n + cs - 1) / cs + 63) / 64 * 64;
        SmallParams p;
        if (sl > kMaxChunks * 64 || small_layout(s, cs, sl, &p) > kSmallSmem) continue;
        if (cs == 16 && !sixteen_fit()) continue;
        if (cs < 8 && sl > 64 && (int64_t)s.G * cs * 4 <= num_sms()) continue;
        *slice = sl;
        return cs;
    }
    return 0;
}

// The rest of a launch's plan from its cluster and slice, and a block's shared memory.
size_t small_plan(const NewtonShape &s, SmallParams *p)
{
    p->m = s.m; p->n = s.n;
    // More than half an SM's shared memory: two blocks on one SM would wait for each other's
    // tensor memory, and two clusters that each hold what the other waits for would never end.
    const size_t smem = std::max<size_t>(small_layout(s, p->cluster, p->slice, p), 120 * 1024);
    // items of the sweep a thread has, at most, against the room for them
    const int V = s.cols % 4 == 0 ? 4 : 1, rows = s.tall ? p->slice : s.m, wide = s.tall ? s.m : std::min(p->slice, s.n);
    int lpr = 1;
    while (lpr < 32 && lpr * V < wide) lpr <<= 1;
    const int64_t items = (int64_t)((rows + kSmallThreads / lpr - 1) / (kSmallThreads / lpr)) * ((wide + lpr * V - 1) / (lpr * V));
    const int64_t kept = items * kSmallThreads * V * 4;
    p->keep = kept <= (int64_t)smem - 1024 - p->oA;
    p->ordered = p->cluster > 1 && p->keep && p->oA + kept > p->oR;
    return smem;
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
    p.in = in; p.out = out; p.steps = steps;
    p.cluster = small_cluster(s, &p.slice);
    p.err = err; p.wait_ns = (uint64_t)wait_limit();
    for (int k = 0; k < 3 * steps; ++k) p.coeffs[k] = coeffs ? coeffs[k] : kNewtonCoeffs[k % 3];
    const bool vec = s.cols % 4 == 0;
    const size_t smem = small_plan(s, &p);
    static bool attr[64][2] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GCONV_ERR_CUDA;
    auto fn = vec ? newton_small_kernel<4> : newton_small_kernel<1>;
    if (!attr[dev][vec]) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmallSmem) != cudaSuccess ||
            cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return GCONV_ERR_CUDA;
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
