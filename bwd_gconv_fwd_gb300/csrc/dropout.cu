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

#include <climits>

namespace gconv {

namespace {

constexpr int kDropThreads = 256;

struct DropArgs {
    const void *x, *res;
    void *y;
    const unsigned long long *rng;
    int64_t count;
    unsigned int bound;          // kept from this on
    int none;                    // p = 1: nothing is kept
    float scale;
};

__device__ __forceinline__ uint4 philox(uint64_t block, uint64_t step, uint64_t seed)
{
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)step, c3 = (uint32_t)(step >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    #pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = (uint64_t)0xD2511F53u * c0, q = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
        c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)q;
        c3 = (uint32_t)p;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

template <typename T> __device__ __forceinline__ T rounded(float v);
template <> __device__ __forceinline__ float rounded<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V elements a thread: 16 bytes where VEC, else four, one by one.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const DropArgs a)
{
    constexpr int V = VEC ? 16 / (int)sizeof(T) : 4;
    const int64_t e = ((int64_t)blockIdx.x * kDropThreads + threadIdx.x) * V;
    if (e >= a.count) return;
    ptx::griddep_wait();
    const T *x = static_cast<const T *>(a.x) + e, *res = a.res ? static_cast<const T *>(a.res) + e : nullptr;
    T *y = static_cast<T *>(a.y) + e;
    const bool whole = VEC && e + V <= a.count;
    Pack<T, V> v, r;
    if (whole) {
        v = *reinterpret_cast<const Pack<T, V> *>(x);
        if (res) r = *reinterpret_cast<const Pack<T, V> *>(res);
    } else {
        #pragma unroll
        for (int j = 0; j < V; ++j)
            if (e + j < a.count) {
                v.v[j] = x[j];
                if (res) r.v[j] = res[j];
            }
    }
    const uint64_t seed = a.rng[0], step = a.rng[1];
    Pack<T, V> o;
    #pragma unroll
    for (int b = 0; b < V / 4; ++b) {
        const uint4 w = philox((uint64_t)e / 4 + b, step, seed);
        const uint32_t word[4] = {w.x, w.y, w.z, w.w};
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool keep = word[j] >= a.bound && !a.none;
            float f = keep ? to_f(v.v[4 * b + j]) * a.scale : 0.f;
            if (res) f += to_f(r.v[4 * b + j]);
            o.v[4 * b + j] = rounded<T>(f);
        }
    }
    if (whole) {
        *reinterpret_cast<Pack<T, V> *>(y) = o;
    } else {
        #pragma unroll
        for (int j = 0; j < V; ++j)
            if (e + j < a.count) y[j] = o.v[j];
    }
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
    const bool vec = on(x, 16) && on(y, 16) && on(res, 16);
    const int64_t per = kDropThreads * (vec ? (int64_t)(16 / es) : 4), grid = (count + per - 1) / per;
    if (grid > INT_MAX) return GCONV_ERR_INVALID_ARG;
    auto *kernel = dtype == GCONV_BF16 ? (vec ? dropout_kernel<__nv_bfloat16, true> : dropout_kernel<__nv_bfloat16, false>)
                                       : (vec ? dropout_kernel<float, true> : dropout_kernel<float, false>);
    launch_dependent(kernel, (unsigned)grid, (unsigned)kDropThreads, 0, static_cast<cudaStream_t>(stream), a);
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
