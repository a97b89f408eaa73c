// dropout.cu -- dropout whose mask is made again instead of stored.
//
//   y = keep x / (1 - p) (+ res),   keep[e] = word e % 4 of Philox-4x32-10 at (e / 4, step), key seed, >= p 2^32
//
// (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011.)  Two or three tensors go
// through once; ten rounds of two 32 x 32 -> 64 bit products make the numbers of four elements, about 12 instructions an
// element, which memory's time covers.  seed and step are read from the device, so that a captured call draws new
// masks when the program moves the step between replays.
#include "internal.h"
#include "ptx.cuh"

#include <algorithm>
#include <climits>

namespace gconv {

namespace {

constexpr int kDropThreads = 256, kDropBlocks = 4;      // threads of a block, blocks an SM

struct DropArgs {
    const void *x, *res;
    void *y;
    const unsigned long long *rng;
    int64_t count;
    unsigned int bound;          // kept from this on
    int none;                    // p = 1: nothing is kept
    float scale;
};

template <typename T> __device__ __forceinline__ T rounded(float v);
template <> __device__ __forceinline__ float rounded<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ void store2(float *to, float x, float y) { to[0] = x; to[1] = y; }
__device__ __forceinline__ void store2(__nv_bfloat16 *to, float x, float y)
{
    *reinterpret_cast<__nv_bfloat162 *>(to) = __floats2bfloat162_rn(x, y);
}

// Keeps a value that is the same in all lanes where the compiler can tell: arithmetic on it is done once a warp.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_or_sync(~0u, v); }

// The numbers of B blocks of four elements side by side, a round's key once.
template <int B>
__device__ __forceinline__ void philox(const uint64_t (&block)[B], uint32_t s0, uint32_t s1, uint32_t k0, uint32_t k1, uint32_t (&w)[B][4])
{
    #pragma unroll
    for (int b = 0; b < B; ++b) {
        w[b][0] = (uint32_t)block[b];
        w[b][1] = (uint32_t)(block[b] >> 32);
        w[b][2] = s0;
        w[b][3] = s1;
    }
    #pragma unroll
    for (int round = 0; round < 10; ++round) {
        #pragma unroll
        for (int b = 0; b < B; ++b) {
            const uint64_t p = (uint64_t)0xD2511F53u * w[b][0], q = (uint64_t)0xCD9E8D57u * w[b][2];
            w[b][0] = (uint32_t)(q >> 32) ^ w[b][1] ^ k0;
            w[b][2] = (uint32_t)(p >> 32) ^ w[b][3] ^ k1;
            w[b][1] = (uint32_t)q;
            w[b][3] = (uint32_t)p;
        }
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

// Elements e .. e + 3, one by one.
template <typename T>
__device__ __forceinline__ void drop_four(const DropArgs &a, int64_t e, uint32_t s0, uint32_t s1, uint32_t k0, uint32_t k1)
{
    const uint64_t block[1] = {(uint64_t)e / 4};
    uint32_t w[1][4];
    philox<1>(block, s0, s1, k0, k1, w);
    #pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (e + j >= a.count) continue;
        const bool keep = w[0][j] >= a.bound && !a.none;
        const float z = keep ? to_f(static_cast<const T *>(a.x)[e + j]) : 0.f;
        const float f = a.res ? fmaf(z, a.scale, to_f(static_cast<const T *>(a.res)[e + j])) : z * a.scale;
        static_cast<T *>(a.y)[e + j] = rounded<T>(f);
    }
}

// A tile is two runs of 16 bytes a thread, a block's width apart.  Blocks stay for all their tiles and ask for the next one's
// elements before they make this one's numbers: the products of ten rounds take 30 us for 51 million elements, about as long as
// their bytes, and without that (a block a tile) the two times add up: 61 us for the 52 measured, 68 for 64 with res.
template <typename T, bool RES>
__global__ void __launch_bounds__(kDropThreads, kDropBlocks) dropout_kernel(const __grid_constant__ DropArgs a)
{
    constexpr int V = 16 / (int)sizeof(T), B = 2 * V / 4;
    constexpr int64_t STEP = kDropThreads * V, TILE = 2 * STEP;
    ptx::griddep_wait();
    const int64_t tiles = a.count / TILE, ahead = (int64_t)gridDim.x * TILE;
    int64_t e = (int64_t)blockIdx.x * TILE + threadIdx.x * V;
    const T *x = static_cast<const T *>(a.x) + e, *res = static_cast<const T *>(a.res) + e;
    T *y = static_cast<T *>(a.y) + e;
    Pack<T, V> v[2], r[2];
    auto load = [&]() {
        #pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[i] = *reinterpret_cast<const Pack<T, V> *>(x + i * STEP);
            if (RES) r[i] = *reinterpret_cast<const Pack<T, V> *>(res + i * STEP);
        }
    };
    if (blockIdx.x < tiles) load();
    const uint64_t seed = a.rng[0], step = a.rng[1];
    const uint32_t k0 = uniform((uint32_t)seed), k1 = uniform((uint32_t)(seed >> 32));
    const uint32_t s0 = uniform((uint32_t)step), s1 = uniform((uint32_t)(step >> 32));
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        uint64_t block[B];
        uint32_t w[B][4];
        #pragma unroll
        for (int b = 0; b < B; ++b) block[b] = ((uint64_t)e + b / (V / 4) * STEP) / 4 + b % (V / 4);
        Pack<T, V> v0[2], r0[2];
        #pragma unroll
        for (int i = 0; i < 2; ++i) { v0[i] = v[i]; r0[i] = r[i]; }
        x += ahead;
        res += ahead;
        if (tile + gridDim.x < tiles) load();
        philox<B>(block, s0, s1, k0, k1, w);
        #pragma unroll
        for (int i = 0; i < 2; ++i) {
            Pack<T, V> o;
            #pragma unroll
            for (int j = 0; j < V; j += 2) {
                float f[2];
                #pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool keep = w[i * (V / 4) + j / 4][j % 4 + h] >= a.bound && !a.none;
                    const float z = keep ? to_f(v0[i].v[j + h]) : 0.f;
                    f[h] = RES ? fmaf(z, a.scale, to_f(r0[i].v[j + h])) : z * a.scale;
                }
                store2(o.v + j, f[0], f[1]);
            }
            *reinterpret_cast<Pack<T, V> *>(y + i * STEP) = o;
        }
        y += ahead;
        e += ahead;
    }
    // what is behind the last whole tile
    for (e = tiles * TILE + ((int64_t)blockIdx.x * kDropThreads + threadIdx.x) * 4; e < a.count; e += (int64_t)gridDim.x * kDropThreads * 4)
        drop_four<T>(a, e, s0, s1, k0, k1);
}

// Tensors off 16 bytes, and small ones: four elements a thread.
template <typename T>
__global__ void __launch_bounds__(kDropThreads) dropout_few_kernel(const __grid_constant__ DropArgs a)
{
    const int64_t e = ((int64_t)blockIdx.x * kDropThreads + threadIdx.x) * 4;
    if (e >= a.count) return;
    ptx::griddep_wait();
    const uint64_t seed = a.rng[0], step = a.rng[1];
    drop_four<T>(a, e, (uint32_t)step, (uint32_t)(step >> 32), (uint32_t)seed, (uint32_t)(seed >> 32));
}


bool on(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

gconv_status dropout(long long count, gconv_dtype dtype, const void *x, const void *res, void *y, const long long *rng,
                     double p, void *stream)
{
    if ((dtype != GCONV_F32 && dtype != GCONV_BF16) || count < 0 || count > (1ll << 40) || !(p >= 0.0 && p <= 1.0))
        return GCONV_ERR_INVALID_ARG;
    if (count == 0) return GCONV_OK;
    const size_t es = dtype == GCONV_BF16 ? 2 : 4;
    if (!x || !y || !rng || !on(rng, 8) || !on(x, es) || !on(y, es) || !on(res, es)) return GCONV_ERR_INVALID_ARG;
    DropArgs a{x, res, y, reinterpret_cast<const unsigned long long *>(rng), count, 0u, 0, 0.f};
    const double bound = p * 4294967296.0;
    if (bound >= 4294967296.0) a.none = 1;
    else {
        a.bound = (unsigned int)bound;
        a.scale = (float)(4294967296.0 / (4294967296.0 - a.bound));
    }
    // From a tile an SM on, blocks that stay: 1.6 us at 622592 elements in bf16 (1.8 with res), 2.2 by four elements a thread; at a
    // quarter of that 1.5 (1.7) and 1.4.  In fp32 1.3 and 1.9 at 311296, 1.2 and 1.5 at a quarter: it would pay there earlier.
    const bool vec = on(x, 16) && on(y, 16) && on(res, 16);
    const int64_t tile = 2 * kDropThreads * (int64_t)(16 / es), tiles = count / tile;
    const int64_t few = (count + 4 * kDropThreads - 1) / (4 * kDropThreads);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (vec && tiles >= num_sms()) {
        auto *kernel = dtype == GCONV_BF16 ? (res ? dropout_kernel<__nv_bfloat16, true> : dropout_kernel<__nv_bfloat16, false>)
                                           : (res ? dropout_kernel<float, true> : dropout_kernel<float, false>);
        launch_dependent(kernel, (unsigned)std::min<int64_t>(tiles, (int64_t)num_sms() * kDropBlocks), (unsigned)kDropThreads, 0, st, a);
    } else {
        if (few > INT_MAX) return GCONV_ERR_INVALID_ARG;
        launch_dependent(dtype == GCONV_BF16 ? dropout_few_kernel<__nv_bfloat16> : dropout_few_kernel<float>, (unsigned)few,
                         (unsigned)kDropThreads, 0, st, a);
    }
    return cudaGetLastError() == cudaSuccess ? GCONV_OK : GCONV_ERR_CUDA;
}

}  // namespace

}  // namespace gconv

using namespace gconv;

extern "C" {

gconv_status gconv_dropout_fwd(long long count, gconv_dtype dtype, const void *x, const void *res, const long long *rng, double p,
                               void *y, void *stream)
{
    return dropout(count, dtype, x, res, y, rng, p, stream);
}

gconv_status gconv_dropout_bwd(long long count, gconv_dtype dtype, const void *dy, const long long *rng, double p, void *dx,
                               void *stream)
{
    return dropout(count, dtype, dy, nullptr, dx, rng, p, stream);
}

}  // extern "C"
