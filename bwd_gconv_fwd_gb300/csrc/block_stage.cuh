// block_stage.cuh -- the block norm / join kernels for groups whose tiles fit in shared memory
// twice (or once): while a block computes one tile, the next lands by asynchronous copies.
//
// These operators do 4 to 40 operations an element against 4 to 16 bytes, so the memory is the
// limit as long as enough of it is in flight: a whole tile of every input here (40 to 200 KB an
// SM), where loads into registers end with each tile's reduction.  Where planes are multiples of 16
// bytes and a channel's share of a tile 64 bytes or more, a tile of a tensor is a few boxes of a
// tensor map, and whole rows are one bulk copy: one thread starts them.  Else the threads copy
// aligned 16-byte pieces, each channel from the boundary before its positions, and read it from
// where they start.  (Such pieces take the threads' own time: a tenth of the
// instructions at 27 x 27, a third while a power of two of threads took a channel and ends were checked
// piece by piece, 39 us there and 35.  Boxes of 32 bytes a row and bulk copies of one
// channel each are slower still: norm of [42,728,28,28] 64 us against 42, gradients at 7 x 7 48 against 33.)
// What is left is the number of instructions, so two positions go through each arithmetic
// instruction (packed fp32 pairs) and every index is 32 bits and steps by constants.
//
// Two forms of a tile: PT positions of every channel of Z rows, or (flat) Z whole rows, which are
// one run of memory, for planes of at most 64 positions.  A thread holds 32 elements (16 where VEC
// is below 4): VEC neighbouring positions (as many as divide P, at most 16 bytes) of 32 / VEC
// channels, so that an address, a predicate and a channel's weight serve VEC elements; where P is
// odd, two neighbours read one by one of 8 channels (VEC = 1).  A thread whose share has fewer channels reads zeros kept
// at the end of each staged tensor instead of branching.
#pragma once

#include "block_norm.cuh"

namespace gconv {

// Elements a thread holds of a tile, and threads of a block, at most.  What a thread does for a tile
// beside its elements (two column sums, places, barriers) is most of the time when it has few: the
// gradient of a join of [64,256,56,56] bf16 took 365 us with 8 in 1024 threads, 214 with 16 in 512 and 196 with 32 in 256.
constexpr int stage_elements(int vec) { return vec >= 4 ? 32 : 16; }
constexpr int stage_threads(int vec) { return vec >= 4 ? 256 : 512; }
constexpr int stage_pairs(int vec) { return vec > 1 ? vec / 2 : 1; }      // pairs of positions a thread holds
constexpr int stage_nch(int vec) { return stage_elements(vec) / 2 / stage_pairs(vec); }   // channels
// Whether a thread's loops run over all the channels it can hold even where it has at most half: with four,
// the branch costs more than it saves (gradient of a join of [64,128,56,56] bf16 in 32 groups 83 us
// without, 90 with); with eight it is a third (the same at 55 x 55 194 and 143, [64,64,112,112] fp32 320 and 267).
constexpr bool whole_share(int nch) { return nch <= 4; }
constexpr uint64_t kStageDrainNs = 1000000000ull;
constexpr int kStageZeros = 32;                                          // bytes of zeros behind a staged tensor


// ---- pairs of fp32 ------------------------------------------------------------------

struct F2 { uint64_t v; };

__device__ __forceinline__ F2 f2(float x, float y)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 parts(F2 a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// 1 / (1 + e^-z) of both: the error is that of the base-2 exponential's and the reciprocal's
// approximations, a few units in the last place.  (Constants stand in single instructions, which
// take them as immediates; a pair would need registers for them.)
__device__ __forceinline__ float sigmoid1(float z)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(e + 1.f));
    return e;
}
__device__ __forceinline__ F2 sigmoid2(F2 z)
{
    const float2 t = parts(z);
    return f2(sigmoid1(t.x), sigmoid1(t.y));
}
__device__ __forceinline__ F2 one_minus(F2 s)
{
    const float2 t = parts(s);
    return f2(1.f - t.x, 1.f - t.y);
}

// What a full gate does: a template argument, so that the arithmetic is straight-line code.
enum { kGateOff = 0, kGateSilu = 1, kGateOther = 2 };   // off: none, or one a channel

// s, from which the gate's value and derivative follow: the sigmoid of z, or z where act is none.
template <int GATE>
__device__ __forceinline__ F2 gate_core(F2 z, bool plain)
{
    const F2 s = sigmoid2(z);
    return GATE == kGateOther && plain ? z : s;
}

// ---- tiles --------------------------------------------------------------------------

// A group too wide for one block's threads and shared memory is dealt over a cluster: block `rank`
// has channels rank Cc, ... of every tile, and the blocks exchange their column sums.  (Z is 1 then.)
struct Part {
    int rank, c0, n;          // first channel of the group, how many
    __device__ __forceinline__ explicit Part(const BlockArgs &a)
    {
        rank = a.cluster > 1 ? (int)ptx::cluster_rank() : 0;
        c0 = rank * a.Cc;
        n = min(a.Cc, a.Cg - c0);
    }
};

// A tile: Z rows from row0, PT positions from p0.
struct Tile {
    int row0, p0;
    __device__ __forceinline__ void set(const BlockArgs &a, int t) { row0 = t / a.tiles * a.Z; p0 = t % a.tiles * a.PT; }
    __device__ __forceinline__ void next(const BlockArgs &a)
    {
        p0 += a.PT;
        if (p0 >= a.P) { p0 = 0; row0 += a.Z; }
    }
};

// What a thread copies where a tile is in pieces: piece k of channels c, c + step, ...
struct Place {
    int k, c, step;
    __device__ __forceinline__ explicit Place(const BlockArgs &a)
    {
        const int n = max(a.pieces, 1);
        step = blockDim.x / n;
        c = threadIdx.x / n;
        k = threadIdx.x - c * n;
        if (c >= step) c = 1 << 30;   // threads left over: no channel is theirs
    }
};

// Starts the copies of one tile of NT tensors to `dst` (a.tensor bytes each; a null tensor is
// skipped).  Boxes and runs complete `full`, at which every thread arrives; pieces are the threads' own.
// A thread whose wait gave up (`ok`) arrives at no barrier again, for the phase it did not see end may still
// be open.
template <typename T, int NT>
__device__ __forceinline__ void stage_tile(const BlockArgs &a, const StageMaps &maps, const Part &g, const Place &pl, const Tile &w,
                                           const char *const (&src)[NT], uint8_t *dst, uint64_t *full, bool ok)
{
    constexpr int es = (int)sizeof(T);
    const uint32_t bar = ptx::smem_u32(full), to0 = ptx::smem_u32(dst);
    const int rows = min(a.Z, a.rows - w.row0) * g.n;          // channels
    const int64_t first = ((int64_t)w.row0 * a.Cg + g.c0) * a.P * es;
    if (a.pieces > 0) {
        // aligned 16-byte pieces, a.pieces threads a channel; a piece that the tensor's end cuts is read up to it
        const int len = min(a.PT, a.P - w.p0) * es;
        const int64_t hop = (int64_t)pl.step * a.P * es;
        const bool cut = first + ((int64_t)rows * a.P + w.p0) * es + 16 > a.bytes;   // the tensor may end in this tile
        int64_t at = first + ((int64_t)pl.c * a.P + w.p0) * es;
        uint32_t to = to0 + (uint32_t)pl.c * (uint32_t)a.pitch + 16u * pl.k;
        #pragma unroll 2
        for (int c = pl.c; c < rows; c += pl.step, at += hop, to += pl.step * a.pitch) {
            const int off = 16 * pl.k - (int)((uint32_t)at & 15u);   // of the piece, from the channel's first position
            if (off >= len) continue;
            const int64_t from = at + off;
            const uint32_t n = cut ? (uint32_t)min((int64_t)16, a.bytes - from) : 16u;
            #pragma unroll
            for (int i = 0; i < NT; ++i)
                if (src[i]) ptx::cp_async16(to + i * a.tensor, src[i] + from, n);
        }
        ptx::cp_async_commit();
        return;
    }
    if (!ok) return;
    uint32_t bytes = 0;
    if (threadIdx.x == 0 && a.boxes > 0) {
        #pragma unroll
        for (int i = 0; i < NT; ++i)
            if (src[i])
                for (int k = 0; k < a.boxes; ++k) {
                    ptx::tma_load_2d(to0 + i * a.tensor + k * a.box_bytes, &maps.m[i], w.p0, w.row0 * a.Cg + g.c0 + k * a.box_rows, bar);
                    bytes += a.box_bytes;
                }
    } else if (threadIdx.x == 0) {
        // one run of memory, widened to 16-byte boundaries; what of the last piece of a tensor is past its
        // end is not read, what is before it goes element by element
        const int64_t lo = first & ~(int64_t)15, end = (first + (int64_t)rows * a.P * es + 15) & ~(int64_t)15;
        const int64_t stop = end <= a.bytes ? end : a.bytes & ~(int64_t)15;
        #pragma unroll
        for (int i = 0; i < NT; ++i)
            if (src[i]) {
                if (stop > lo) {
                    ptx::bulk_g2s(to0 + i * a.tensor, src[i] + lo, (uint32_t)(stop - lo), bar);
                    bytes += (uint32_t)(stop - lo);
                }
                for (int64_t at = max(lo, stop); end > a.bytes && at < a.bytes; at += es)
                    *reinterpret_cast<T *>(dst + i * a.tensor + (int)(at - lo)) = *reinterpret_cast<const T *>(src[i] + at);
            }
    }
    ptx::mbar_arrive_expect_tx(bar, bytes);
}

// A thread's positions of a staged channel (a shared-memory address: 32 bits, an offset in the
// instruction), and their store to a tensor.
__device__ __forceinline__ F2 pair_of(uint32_t two_bf16)
{
    return f2(__uint_as_float(two_bf16 << 16), __uint_as_float(two_bf16 & 0xffff0000u));
}

template <typename T, int VEC>
__device__ __forceinline__ void read_vec(uint32_t at, F2 (&v)[stage_pairs(VEC)])
{
    constexpr int words = VEC * (int)sizeof(T) / 4;   // 32-bit words, where the positions are aligned
    if constexpr (VEC == 1 && sizeof(T) == 2) {
        uint16_t a, b;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(a) : "r"(at));
        asm volatile("ld.shared.u16 %0, [%1+2];" : "=h"(b) : "r"(at));
        v[0] = f2(__uint_as_float((uint32_t)a << 16), __uint_as_float((uint32_t)b << 16));
    } else if constexpr (VEC == 1) {
        float a, b;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(a) : "r"(at));
        asm volatile("ld.shared.f32 %0, [%1+4];" : "=f"(b) : "r"(at));
        v[0] = f2(a, b);
    } else {
        uint32_t w[words];
        if constexpr (words == 4)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
        else if constexpr (words == 2)
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
        else
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at));
        #pragma unroll
        for (int k = 0; k < VEC / 2; ++k)
            v[k] = sizeof(T) == 2 ? pair_of(w[k]) : f2(__uint_as_float(w[(2 * k) % words]), __uint_as_float(w[(2 * k + 1) % words]));
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void write_vec(void *p, uint32_t i, const F2 (&v)[stage_pairs(VEC)], bool ok0, bool ok1)
{
    if constexpr (VEC == 1) {
        const float2 f = parts(v[0]);
        T *q = static_cast<T *>(p) + i;
        if (ok0) from_f(f.x, q);
        if (ok1) from_f(f.y, q + 1);
    } else {
        Pack<T, VEC> o;
        #pragma unroll
        for (int k = 0; k < VEC / 2; ++k) {
            const float2 f = parts(v[k]);
            if constexpr (sizeof(T) == 2) reinterpret_cast<__nv_bfloat162 *>(&o)[k] = __floats2bfloat162_rn(f.x, f.y);
            else { o.v[2 * k] = f.x; o.v[2 * k + 1] = f.y; }
        }
        if (ok0) *reinterpret_cast<Pack<T, VEC> *>(static_cast<T *>(p) + i) = o;
    }
}

__device__ __forceinline__ F2 shfl_xor2(F2 v, int m)
{
    const float2 f = parts(v);
    return f2(__shfl_xor_sync(0xffffffffu, f.x, m), __shfl_xor_sync(0xffffffffu, f.y, m));
}

// Adds N values over the lanes that differ in the bits 16, ..., TX: a lane keeps half of its values at
// each level while it has two, and stores what it ends with as values base.. of its vector tx.
template <int TX, int N, int M = 16>
__device__ __forceinline__ void scatter_sum(const F2 (&v)[N], uint64_t *to, int tx, int base)
{
    if constexpr (M < TX || M == 0) {
        #pragma unroll
        for (int i = 0; i < N; ++i) to[(base + i) * TX + tx] = v[i].v;
    } else if constexpr (N > 1) {
        const bool high = threadIdx.x & M;
        F2 keep[N / 2];
        #pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const F2 mine = high ? v[N / 2 + i] : v[i], theirs = high ? v[i] : v[N / 2 + i];
            keep[i] = add2(mine, shfl_xor2(theirs, M));
        }
        scatter_sum<TX, N / 2, M / 2>(keep, to, tx, base + (high ? N / 2 : 0));
    } else {
        const F2 sum[1] = {add2(v[0], shfl_xor2(v[0], M))};
        scatter_sum<TX, 1, M / 2>(sum, to, tx, base);
    }
}

__device__ __forceinline__ F2 shfl2(F2 v, int lane)
{
    const float2 f = parts(v);
    return f2(__shfl_sync(0xffffffffu, f.x, lane), __shfl_sync(0xffffffffu, f.y, lane));
}

// From the sum of squares of both positions r = 1 / sqrt(mean + eps), and from the sum of g w t
// m = -mean(g w t) r^3, a factor at a time: r^3 alone leaves fp32 where r is beyond 1e-13 .. 1e13.
__device__ __forceinline__ F2 root2(const BlockArgs &a, F2 sum)
{
    const float2 s = parts(sum);
    return f2(rsqrtf(fmaf(s.x, a.inv_cg, a.eps)), rsqrtf(fmaf(s.y, a.inv_cg, a.eps)));
}
__device__ __forceinline__ F2 pull2(const BlockArgs &a, F2 sum, F2 r) { return mul2(mul2(mul2(mul2(sum, f2(-a.inv_cg)), r), r), r); }

// Adds v over the TY threads that share a row and a vector and turns the sums into r (the first
// NP) and m (the second NP, with TWO), the same bits in every thread: within a warp by shuffles
// that split the values among its lanes, then over a row's warps through shared memory, where
// every warp adds all of its row's sums, a lane a few of them, and hands them round: one block
// barrier in all.  In a cluster a row's first warp sends its block's sums to the other blocks, and every
// warp adds those in rank order.  `red`: two halves (`turn`: a half is written again only two
// barriers after it was read), each N TX pairs a warp, and behind them the same for the cluster's blocks.
template <int NP, bool TWO, int TX>
__device__ __forceinline__ void column_roots_tx(F2 (&v)[TWO ? 2 * NP : NP], float *red, const BlockArgs &a, const Part &g,
                                                int &turn, int tx, int ty, int z)
{
    constexpr int N = TWO ? 2 * NP : NP, width = N * TX, half = NP * TX, slots = (half + 31) / 32;
    const int lane = threadIdx.x & 31, warps = a.TY / (32 / TX), in_row = ty * TX + tx;
    uint64_t *base = reinterpret_cast<uint64_t *>(red);
    uint64_t *mine = base + (turn * a.Z + z) * warps * width;
    scatter_sum<TX, N>(v, mine + (in_row >> 5) * width, tx, 0);
    __syncthreads();
    const int at = half >= 32 ? lane : lane % half;          // value (and sum of g w t `half` on) of this lane
    F2 s[slots], u[slots];
    #pragma unroll
    for (int k = 0; k < slots; ++k) {
        s[k] = F2{mine[at + 32 * k]};
        u[k] = F2{TWO ? mine[half + at + 32 * k] : 0};
    }
    #pragma unroll 4
    for (int w = 1; w < warps; ++w)
        #pragma unroll
        for (int k = 0; k < slots; ++k) {
            s[k] = add2(s[k], F2{mine[w * width + at + 32 * k]});
            if constexpr (TWO) u[k] = add2(u[k], F2{mine[w * width + half + at + 32 * k]});
        }
    if (a.cluster > 1) {
        uint64_t *others = base + 2 * warps * width + turn * a.cluster * width;
        if (in_row < 32 && lane < (half < 32 ? half : 32))
            for (int k = 0; k < a.cluster; ++k)
                #pragma unroll
                for (int q = 0; q < slots; ++q) {
                    const uint32_t to = ptx::map_to(ptx::smem_u32(others + g.rank * width + at + 32 * q), (uint32_t)k);
                    ptx::st_cluster64(to, s[q].v);
                    if constexpr (TWO) ptx::st_cluster64(to + half * 8, u[q].v);
                }
        __syncwarp();
        ptx::cluster_sync();
        #pragma unroll
        for (int q = 0; q < slots; ++q) {
            s[q] = F2{others[at + 32 * q]};
            u[q] = F2{TWO ? others[half + at + 32 * q] : 0};
            for (int k = 1; k < a.cluster; ++k) {
                s[q] = add2(s[q], F2{others[k * width + at + 32 * q]});
                if constexpr (TWO) u[q] = add2(u[q], F2{others[k * width + half + at + 32 * q]});
            }
        }
    }
    turn ^= 1;
    #pragma unroll
    for (int k = 0; k < slots; ++k) {
        s[k] = root2(a, s[k]);
        if constexpr (TWO) u[k] = pull2(a, u[k], s[k]);
    }
    #pragma unroll
    for (int i = 0; i < NP; ++i) {   // value i of vector tx is number i TX + tx
        const int from = (i * TX + tx) & 31, slot = i * TX / 32;
        v[i] = TX == 32 ? s[slot] : shfl2(s[slot], from);
        if constexpr (TWO) v[NP + i] = TX == 32 ? u[slot] : shfl2(u[slot], from);
    }
}

template <int NP, bool TWO>
__device__ __forceinline__ void column_roots(F2 (&v)[TWO ? 2 * NP : NP], float *red, const BlockArgs &a, const Part &g, int &turn,
                                             int tx, int ty, int z)
{
    constexpr int N = TWO ? 2 * NP : NP;
    const int per_row = a.TX * a.TY;
    if (per_row <= 32 && a.cluster == 1) {
        for (int m = a.TX; m < per_row; m <<= 1) {
            #pragma unroll
            for (int i = 0; i < N; ++i) v[i] = add2(v[i], shfl_xor2(v[i], m));
        }
        #pragma unroll
        for (int i = 0; i < NP; ++i) {
            v[i] = root2(a, v[i]);
            if constexpr (TWO) v[NP + i] = pull2(a, v[NP + i], v[i]);
        }
        return;
    }
    switch (a.TX) {
    case 32: column_roots_tx<NP, TWO, 32>(v, red, a, g, turn, tx, ty, z); break;
    case 16: column_roots_tx<NP, TWO, 16>(v, red, a, g, turn, tx, ty, z); break;
    case 8: column_roots_tx<NP, TWO, 8>(v, red, a, g, turn, tx, ty, z); break;
    case 4: column_roots_tx<NP, TWO, 4>(v, red, a, g, turn, tx, ty, z); break;
    case 2: column_roots_tx<NP, TWO, 2>(v, red, a, g, turn, tx, ty, z); break;
    default: column_roots_tx<NP, TWO, 1>(v, red, a, g, turn, tx, ty, z); break;
    }
}

// Zeros at the end of each staged tensor, and in the whole of the first where it has no source.
template <int NT>
__device__ __forceinline__ void stage_zeros(const BlockArgs &a, uint8_t *smem, bool first)
{
    constexpr int words = kStageZeros / 4;
    for (int i = threadIdx.x; i < a.stages * NT * words; i += blockDim.x)
        *reinterpret_cast<uint32_t *>(smem + (i / words + 1) * a.tensor - kStageZeros + (i % words) * 4) = 0;
    if (first)
        for (int s = 0; s < a.stages; ++s)
            for (int i = threadIdx.x * 4; i < a.tensor; i += blockDim.x * 4)
                *reinterpret_cast<uint32_t *>(smem + s * NT * a.tensor + i) = 0;
}

// A thread's place: vector tx, channels ty, ty + TY, ... of row z of the tile, and from it the
// offsets of its first channel and the steps to the next.  (32 bits: the low four bits of a
// byte address survive, and a tensor has fewer than 2^31 elements.)
struct Seat {
    int tx, ty, z, pos, c0;
    int s_first, s_step, m_step;
    uint32_t e_step;
};

template <typename T, int VEC>
__device__ __forceinline__ Seat seat(const BlockArgs &a, const Part &g)
{
    constexpr int es = (int)sizeof(T);
    Seat s;
    s.tx = threadIdx.x % a.TX;
    const int ry = threadIdx.x / a.TX;
    s.ty = ry % a.TY;
    s.z = ry / a.TY;
    s.pos = (VEC > 1 ? VEC : 2) * s.tx;
    s.c0 = s.z * g.n + s.ty;
    s.s_first = s.c0 * a.pitch + s.pos * es;
    s.s_step = a.TY * a.pitch;
    s.m_step = a.flat ? 0 : a.TY * a.P * es;
    s.e_step = (uint32_t)(a.TY * a.P);
    return s;
}

template <typename T>
__device__ __forceinline__ int staged_at(const BlockArgs &a, const Seat &s, uint32_t m0, int j, bool has)
{
    if (!has) return a.tensor - kStageZeros;
    return s.s_first + j * s.s_step + (int)((m0 + (uint32_t)(j * s.m_step)) & 15u);
}

// Byte offset, modulo 16, of the thread's first channel in this tile (flat: of the tile).
template <typename T>
__device__ __forceinline__ uint32_t misfit(const BlockArgs &a, const Part &g, const Seat &s, const Tile &w)
{
    const uint32_t first = ((uint32_t)w.row0 * (uint32_t)a.Cg + (uint32_t)g.c0) * (uint32_t)a.P;
    return (first + (a.flat ? 0u : (uint32_t)s.c0 * (uint32_t)a.P + (uint32_t)w.p0)) * (uint32_t)sizeof(T);
}

// Adds N values over the TX lanes of a vector: at each level a lane keeps half of its values while it
// has two, so that N and not N log TX values are exchanged; `put` gets each sum once.
template <int N, int M, typename Put>
__device__ __forceinline__ void lane_sums(const float (&v)[N], int TX, int tx, int base, const Put &put)
{
    if constexpr (M == 0) {
        #pragma unroll
        for (int i = 0; i < N; ++i) put(base + i, v[i]);
    } else if (M >= TX) {
        lane_sums<N, M / 2>(v, TX, tx, base, put);
    } else if constexpr (N > 1) {
        const bool high = tx & M;
        float keep[N / 2];
        #pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float mine = high ? v[N / 2 + i] : v[i], theirs = high ? v[i] : v[N / 2 + i];
            keep[i] = mine + __shfl_xor_sync(0xffffffffu, theirs, M);
        }
        lane_sums<N / 2, M / 2>(keep, TX, tx, base + (high ? N / 2 : 0), put);
    } else {
        const float sum[1] = {v[0] + __shfl_xor_sync(0xffffffffu, v[0], M)};
        lane_sums<1, M / 2>(sum, TX, tx, base, put);
    }
}

// Every tile's copies were waited for, unless a wait gave up: then the last ones get the time to land
// before the block's shared memory is another's.  (Pieces are always waited for.)
__device__ __forceinline__ void stage_drain(bool ok)
{
    if (__syncthreads_or(!ok) && threadIdx.x == 0) ptx::let_pass(kStageDrainNs);
    __syncthreads();
}

// The channel numbers of the thread's row: the next norm's weight and the branch's coefficient (times
// the channel gate), 0 where there is no channel.  Every load is issued before the first use, none
// behind a branch of its own.
template <typename T, int NCH, bool POST, bool NEXT>
__device__ __forceinline__ void row_numbers(const BlockArgs &a, const Part &g, const Seat &s, int row, bool in_row,
                                            const bool (&has)[NCH], float (&wn)[NCH], float (&kb)[NCH])
{
    const int ch0 = in_row ? (row % a.G) * a.Cg + g.c0 : 0;
    const int64_t nc0 = in_row ? (int64_t)row * a.Cg + g.c0 : 0;
    int at[NCH];
    float sc[NCH], zc[NCH];
    #pragma unroll
    for (int j = 0; j < NCH; ++j) {
        at[j] = in_row && has[j] ? s.ty + j * a.TY : 0;
        wn[j] = kb[j] = sc[j] = 1.f;
        zc[j] = 0.f;
    }
    if (NEXT && a.w2) {
        #pragma unroll
        for (int j = 0; j < NCH; ++j) wn[j] = a.w2[ch0 + at[j]];
    }
    if (POST && a.w) {
        #pragma unroll
        for (int j = 0; j < NCH; ++j) kb[j] = a.w[ch0 + at[j]];
    }
    if (POST && a.s) {
        #pragma unroll
        for (int j = 0; j < NCH; ++j) sc[j] = a.s[ch0 + at[j]];
    }
    if (POST && a.gate == GCONV_GATE_CHANNEL) {
        #pragma unroll
        for (int j = 0; j < NCH; ++j) zc[j] = to_f(static_cast<const T *>(a.z)[nc0 + at[j]]);
    }
    #pragma unroll
    for (int j = 0; j < NCH; ++j) {
        if (POST) kb[j] = __fmul_rn(kb[j], sc[j]);
        if (POST && a.gate == GCONV_GATE_CHANNEL) kb[j] = __fmul_rn(kb[j], gate_value(zc[j], a.act));
        if (!(in_row && has[j])) wn[j] = kb[j] = 0.f;
    }
}

// Forward.  One sweep over a tile gives sum h^2 a position, the second out (kept in registers) and
// sum out^2, the third next; a norm alone is the first and the third.  Every tensor crosses the
// memory once.  Two blocks an SM, so that one's reductions stand beside the other's sweeps (a join of
// [64,256,56,56] bf16 167 us with one, 117 with two).  Now 103 to 111 us there, 514 MB, 4.6 to 5.0 TB/s
// against the 6.8 of a plain copy: what is left is the sweeps' instructions and the wait of the first and the
// last tile of a block.  (With VEC 1 and 2 a block has 512 threads, so 64 registers each: the joins
// spill 40 to 72 bytes there without `next` and 140 to 168 with it.)
template <typename T, int VEC, bool POST, bool NEXT, int GATE>
__global__ void __launch_bounds__(stage_threads(VEC), 2) block_fwd_stage_kernel(const BlockArgs a, const __grid_constant__ StageMaps maps)
{
    constexpr int NT = POST ? 3 : 1, NP = stage_pairs(VEC), NCH = stage_nch(VEC);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-ptx::smem_u32(smem_raw) & 127u);   // boxes land on 128-byte boundaries
    __shared__ __align__(8) uint64_t bars[2];
    float *red = reinterpret_cast<float *>(smem + a.stages * NT * a.tensor);
    const Part g(a);
    const Place pl(a);
    const Seat s = seat<T, VEC>(a, g);
    constexpr bool full = GATE != kGateOff;
    const bool plain = a.act == GCONV_ACT_NONE;
    const char *src[NT];
    src[0] = static_cast<const char *>(a.x);
    if constexpr (POST) { src[1] = static_cast<const char *>(a.h); src[2] = full ? static_cast<const char *>(a.z) : nullptr; }
    if (threadIdx.x == 0) {
        ptx::mbar_init(ptx::smem_u32(&bars[0]), blockDim.x);
        ptx::mbar_init(ptx::smem_u32(&bars[1]), blockDim.x);
        ptx::fence_mbar_init();
    }
    stage_zeros<NT>(a, smem, !src[0]);
    __syncthreads();
    bool ok = true;
    // Waits for a tile's copies; after a wait that gave up, none waits again.
    auto landed = [&](int t, int t0, int t1) {
        if (a.pieces > 0) {
            // the next tile's pieces, started since, may stay in flight
            if (a.stages == 2 && t + 1 < t1) ptx::cp_async_wait_group<1>();
            else ptx::cp_async_wait_group<0>();
            __syncthreads();
            return;
        }
        const int k = t - t0, buf = k & (a.stages - 1);
        if (ok && !ptx::mbar_wait(ptx::smem_u32(&bars[buf]), (uint32_t)(k / a.stages) & 1u, a.wait_ns)) {
            ok = false;
            raise_device_error(a.err, DEVERR_WAIT_TIMEOUT);
        }
    };
    const int walker = blockIdx.x / a.cluster;
    const int t0 = walker * a.per, t1 = min(a.total, t0 + a.per);
    Tile w, ahead;
    w.set(a, t0);
    ahead = w;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (a.cluster > 1) ptx::cluster_sync();   // the others' shared memory may be written from here on
    stage_tile<T, NT>(a, maps, g, pl, ahead, src, smem, &bars[0], ok);

    int at_row = -1, turn = 0;
    float kb[NCH], wn[NCH];
    bool has[NCH];
    #pragma unroll
    for (int j = 0; j < NCH; ++j) has[j] = s.ty + j * a.TY < g.n;
    const bool wide = whole_share(NCH) || a.TY * (NCH / 2) < g.n;   // more than half of them
    for (int t = t0; t < t1; ++t, w.next(a)) {
        const int buf = (t - t0) & (a.stages - 1);
        if (a.stages == 1 && t > t0) {
            __syncthreads();   // the tile before has been read
            ahead.next(a);
            stage_tile<T, NT>(a, maps, g, pl, ahead, src, smem, &bars[0], ok);
        }
        const bool in_row = w.row0 + s.z < a.rows;
        if (at_row != w.row0) {
            at_row = w.row0;
            row_numbers<T, NCH, POST, NEXT>(a, g, s, at_row + s.z, in_row, has, wn, kb);
        }
        if (a.stages == 2 && t + 1 < t1) {
            if (t > t0) __syncthreads();   // the tile before has been read
            ahead.next(a);
            stage_tile<T, NT>(a, maps, g, pl, ahead, src, smem + (buf ^ 1) * NT * a.tensor, &bars[buf ^ 1], ok);
        }
        landed(t, t0, t1);
        const uint32_t st = ptx::smem_u32(smem) + buf * NT * a.tensor;
        const bool ok0 = in_row && w.p0 + s.pos < a.P, ok1 = in_row && w.p0 + s.pos + 1 < a.P;
        const uint32_t m0 = misfit<T>(a, g, s, w);
        const uint32_t e0 = ((uint32_t)w.row0 * (uint32_t)a.Cg + (uint32_t)(g.c0 + s.c0)) * (uint32_t)a.P + (uint32_t)(w.p0 + s.pos);
        int at[NCH];
        F2 r[NP], o[NCH][NP];
        #pragma unroll
        for (int k = 0; k < NP; ++k) r[k] = f2(0.f);
        #pragma unroll
        for (int j = 0; j < NCH; ++j) {
            if (j == NCH / 2 && !wide) break;
            at[j] = staged_at<T>(a, s, m0, j, has[j]);
            read_vec<T, VEC>(st + (POST ? a.tensor : 0) + at[j], o[j]);
            #pragma unroll
            for (int k = 0; k < NP; ++k) r[k] = fma2(o[j][k], o[j][k], r[k]);
        }
        column_roots<NP, false>(r, red, a, g, turn, s.tx, s.ty, s.z);
        if (POST) {
            F2 sum[NP];
            #pragma unroll
            for (int k = 0; k < NP; ++k) sum[k] = f2(0.f);
            #pragma unroll
            for (int j = 0; j < NCH; ++j) {
                if (j == NCH / 2 && !wide) break;
                    F2 x[NP], z[NP];
                    read_vec<T, VEC>(st + at[j], x);
                    if (full) read_vec<T, VEC>(st + 2 * a.tensor + at[j], z);
                    #pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        F2 kg = f2(kb[j]);
                        if (full) {
                            const F2 sg = gate_core<GATE>(z[k], plain);
                            kg = mul2(kg, GATE == kGateSilu ? mul2(z[k], sg) : sg);
                        }
                        o[j][k] = fma2(kg, mul2(o[j][k], r[k]), x[k]);
                        sum[k] = fma2(o[j][k], o[j][k], sum[k]);
                    }
                    write_vec<T, VEC>(a.out, e0 + j * s.e_step, o[j], has[j] && ok0, has[j] && ok1);
                }
            if (!NEXT) continue;
            column_roots<NP, false>(sum, red, a, g, turn, s.tx, s.ty, s.z);
            #pragma unroll
            for (int k = 0; k < NP; ++k) r[k] = sum[k];
        }
        #pragma unroll
        for (int j = 0; j < NCH; ++j) {
            if (j == NCH / 2 && !wide) break;
            #pragma unroll
            for (int k = 0; k < NP; ++k) o[j][k] = mul2(o[j][k], mul2(r[k], f2(wn[j])));
            write_vec<T, VEC>(a.next, e0 + j * s.e_step, o[j], has[j] && ok0, has[j] && ok1);
        }
    }
    stage_drain(ok);
}

// A pair's sum, without what stands at a dead position.
template <int VEC>
__device__ __forceinline__ F2 live_only(F2 v, bool ok0, bool ok1)
{
    if constexpr (VEC > 1) return ok0 ? v : f2(0.f);
    const float2 f = parts(v);
    return f2(ok0 ? f.x : 0.f, ok1 ? f.y : 0.f);
}

// Backward.  A block walks consecutive tiles; its channel sums of a block of rows stay in
// registers and go to part[i][row][channel] when the rows change, i counting the blocks that
// share those rows: no atomics, so the same bits each time.  Dead positions hold what an earlier tile left: they meet no live one but in
// the channel sums, which leave them out.
//   Measured, each tensor crossing the memory once: join with next norm, [64,256,56,56] bf16, 822 MB,
// 189 us (4.3 TB/s of the 6.8 of a plain copy): five tensors twice in shared memory leave one block
// of 8 warps an SM, too few to hide the sweeps' latency.  Norm of [128,96,27,27] bf16 in 2 groups,
// 72 MB, 35 us (2.1 TB/s): planes of odd size are copied in pieces, read and stored element by
// element, 64 instructions each.  Join of [32,1024,7,7] fp32, 39 MB, 27 us: 128 tiles on 64 clusters of two
// blocks that hold one tile at a time, so that each walks two with copies, sweeps and the cluster's two exchanges in
// turn, and 24 of the SMs have no block.
template <typename T, int VEC, bool POST, bool NEXT, int GATE>
__global__ void __launch_bounds__(stage_threads(VEC), POST ? 1 : 2) block_bwd_stage_kernel(const BlockArgs a, const __grid_constant__ StageMaps maps)
{
    constexpr int NT = POST && NEXT ? 5 : 3, NP = stage_pairs(VEC), NCH = stage_nch(VEC);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-ptx::smem_u32(smem_raw) & 127u);   // boxes land on 128-byte boundaries
    __shared__ __align__(8) uint64_t bars[2];
    float *red = reinterpret_cast<float *>(smem + a.stages * NT * a.tensor);
    const Part g(a);
    const Place pl(a);
    const Seat s = seat<T, VEC>(a, g);
    constexpr bool full = GATE != kGateOff;
    const bool plain = a.act == GCONV_ACT_NONE;
    const char *src[NT];
    src[0] = static_cast<const char *>(a.dout);
    constexpr int iX = 1, iG = 2, iH = NEXT ? 3 : 1, iZ = NEXT ? 4 : 2;
    if constexpr (NEXT) { src[iX] = static_cast<const char *>(a.x); src[iG] = static_cast<const char *>(a.dnext); }
    if constexpr (POST) { src[iH] = static_cast<const char *>(a.h); src[iZ] = full ? static_cast<const char *>(a.z) : nullptr; }
    if (threadIdx.x == 0) {
        ptx::mbar_init(ptx::smem_u32(&bars[0]), blockDim.x);
        ptx::mbar_init(ptx::smem_u32(&bars[1]), blockDim.x);
        ptx::fence_mbar_init();
    }
    stage_zeros<NT>(a, smem, !src[0]);
    __syncthreads();
    bool ok = true;
    // Waits for a tile's copies; after a wait that gave up, none waits again.
    auto landed = [&](int t, int t0, int t1) {
        if (a.pieces > 0) {
            // the next tile's pieces, started since, may stay in flight
            if (a.stages == 2 && t + 1 < t1) ptx::cp_async_wait_group<1>();
            else ptx::cp_async_wait_group<0>();
            __syncthreads();
            return;
        }
        const int k = t - t0, buf = k & (a.stages - 1);
        if (ok && !ptx::mbar_wait(ptx::smem_u32(&bars[buf]), (uint32_t)(k / a.stages) & 1u, a.wait_ns)) {
            ok = false;
            raise_device_error(a.err, DEVERR_WAIT_TIMEOUT);
        }
    };
    const int walker = blockIdx.x / a.cluster;
    const int t0 = walker * a.per, t1 = min(a.total, t0 + a.per);
    const int64_t NC = (int64_t)a.rows * a.Cg;
    Tile w, ahead;
    w.set(a, t0);
    ahead = w;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (a.cluster > 1) ptx::cluster_sync();   // the others' shared memory may be written from here on
    stage_tile<T, NT>(a, maps, g, pl, ahead, src, smem, &bars[0], ok);

    int at_row = -1, turn = 0;
    bool in_row = false;
    F2 acc2[NCH], acck[NCH];
    float wn[NCH], kb[NCH];
    bool has[NCH];
    #pragma unroll
    for (int j = 0; j < NCH; ++j) has[j] = s.ty + j * a.TY < g.n;
    const bool wide = whole_share(NCH) || a.TY * (NCH / 2) < g.n;   // more than half of them
    auto flush = [&] {
        const int share = walker - (int)((int64_t)(at_row / a.Z) * a.tiles / a.per);
        float *p0 = a.part + share * NC + (int64_t)(at_row + s.z) * a.Cg + g.c0 + s.ty;
        float v[2 * NCH];
        #pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const float2 x = parts(acc2[j]), y = parts(acck[j]);
            v[j] = x.x + x.y;
            v[NCH + j] = y.x + y.y;
        }
        lane_sums<2 * NCH, 16>(v, a.TX, s.tx, 0, [&](int n, float sum) {   // number n: of channel n % NCH
            const int c = s.ty + (n % NCH) * a.TY;
            if (!in_row || c >= g.n) return;
            float *to = p0 + (n % NCH) * a.TY;
            if (NEXT && n < NCH) to[0] = sum;
            if (POST && n >= NCH) to[a.splits * NC] = sum;
        });
    };
    for (int t = t0; t < t1; ++t, w.next(a)) {
        const int buf = (t - t0) & (a.stages - 1);
        if (a.stages == 1 && t > t0) {
            __syncthreads();   // the tile before has been read
            ahead.next(a);
            stage_tile<T, NT>(a, maps, g, pl, ahead, src, smem, &bars[0], ok);
        }
        if (at_row != w.row0) {
            if (at_row >= 0) flush();
            at_row = w.row0;
            in_row = w.row0 + s.z < a.rows;
            row_numbers<T, NCH, POST, NEXT>(a, g, s, at_row + s.z, in_row, has, wn, kb);
            #pragma unroll
            for (int j = 0; j < NCH; ++j) acc2[j] = acck[j] = f2(0.f);
        }
        if (a.stages == 2 && t + 1 < t1) {
            if (t > t0) __syncthreads();   // the tile before has been read
            ahead.next(a);
            stage_tile<T, NT>(a, maps, g, pl, ahead, src, smem + (buf ^ 1) * NT * a.tensor, &bars[buf ^ 1], ok);
        }
        landed(t, t0, t1);
        const uint32_t st = ptx::smem_u32(smem) + buf * NT * a.tensor;
        const bool ok0 = in_row && w.p0 + s.pos < a.P, ok1 = in_row && w.p0 + s.pos + 1 < a.P;
        const uint32_t m0 = misfit<T>(a, g, s, w);
        const uint32_t e0 = ((uint32_t)w.row0 * (uint32_t)a.Cg + (uint32_t)(g.c0 + s.c0)) * (uint32_t)a.P + (uint32_t)(w.p0 + s.pos);
        int at[NCH];
        #pragma unroll
        for (int j = 0; j < NCH; ++j) {
            if (j == NCH / 2 && !wide) break;
            at[j] = staged_at<T>(a, s, m0, j, has[j]);
        }
        F2 d[NCH][NP], sum[2 * NP];
        F2 rm[2 * NP];   // r and m
        #pragma unroll
        for (int k = 0; k < 2 * NP; ++k) sum[k] = f2(0.f);
        if (NEXT) {
            #pragma unroll
            for (int j = 0; j < NCH; ++j) {
                if (j == NCH / 2 && !wide) break;
                    F2 x[NP], g[NP];
                    read_vec<T, VEC>(st + iX * a.tensor + at[j], x);
                    read_vec<T, VEC>(st + iG * a.tensor + at[j], g);
                    #pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        sum[k] = fma2(x[k], x[k], sum[k]);
                        sum[NP + k] = fma2(x[k], mul2(g[k], f2(wn[j])), sum[NP + k]);
                    }
                }
            column_roots<NP, true>(sum, red, a, g, turn, s.tx, s.ty, s.z);
            #pragma unroll
            for (int k = 0; k < 2 * NP; ++k) { rm[k] = sum[k]; sum[k] = f2(0.f); }
        }
        F2 sg[NCH][NP];   // the gate's sigmoid, or its value without one
        #pragma unroll
        for (int j = 0; j < NCH; ++j) {
            if (j == NCH / 2 && !wide) break;
                read_vec<T, VEC>(st + at[j], d[j]);
                if (NEXT) {
                    F2 x[NP], g[NP], u = f2(0.f);
                    read_vec<T, VEC>(st + iX * a.tensor + at[j], x);
                    read_vec<T, VEC>(st + iG * a.tensor + at[j], g);
                    #pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        g[k] = mul2(g[k], rm[k]);
                        d[j][k] = fma2(x[k], rm[NP + k], fma2(g[k], f2(wn[j]), d[j][k]));
                        u = fma2(g[k], x[k], u);
                    }
                    acc2[j] = add2(acc2[j], live_only<VEC>(u, ok0, ok1));
                    write_vec<T, VEC>(a.dx, e0 + j * s.e_step, d[j], has[j] && ok0, has[j] && ok1);
                }
                if (POST) {
                    F2 h[NP], z[NP];
                    read_vec<T, VEC>(st + iH * a.tensor + at[j], h);
                    if (full) read_vec<T, VEC>(st + iZ * a.tensor + at[j], z);
                    #pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        F2 v = mul2(d[j][k], f2(kb[j]));
                        if (full) {
                            sg[j][k] = gate_core<GATE>(z[k], plain);
                            v = mul2(v, GATE == kGateSilu ? mul2(z[k], sg[j][k]) : sg[j][k]);
                        }
                        sum[k] = fma2(h[k], h[k], sum[k]);
                        sum[NP + k] = fma2(h[k], v, sum[NP + k]);
                    }
                }
            }
        if (!POST) continue;
        column_roots<NP, true>(sum, red, a, g, turn, s.tx, s.ty, s.z);
        #pragma unroll
        for (int j = 0; j < NCH; ++j) {
            if (j == NCH / 2 && !wide) break;
                const uint32_t e = e0 + j * s.e_step;
                F2 h[NP], z[NP], u = f2(0.f);
                read_vec<T, VEC>(st + iH * a.tensor + at[j], h);
                if (GATE == kGateSilu) read_vec<T, VEC>(st + iZ * a.tensor + at[j], z);
                #pragma unroll
                for (int k = 0; k < NP; ++k) {
                    const F2 dr = mul2(d[j][k], sum[k]), dk = mul2(dr, f2(kb[j]));
                    F2 dh = dk;   // the channel gate is in kb; its own gradient needs the sum without it
                    if (full) {
                        // act'(z): 1; s (1 - s); s (1 + z (1 - s)) = s + g (1 - s)
                        const F2 rest = one_minus(sg[j][k]);
                        const F2 g = GATE == kGateSilu ? mul2(z[k], sg[j][k]) : sg[j][k];
                        const F2 dg = GATE == kGateSilu ? fma2(g, rest, sg[j][k]) : plain ? f2(1.f) : mul2(g, rest);
                        sg[j][k] = mul2(mul2(dk, h[k]), dg);   // dz
                        u = fma2(mul2(dr, h[k]), g, u);
                        dh = mul2(dk, g);
                    } else {
                        u = fma2(dr, h[k], u);
                    }
                    d[j][k] = fma2(h[k], sum[NP + k], dh);
                }
                acck[j] = add2(acck[j], live_only<VEC>(u, ok0, ok1));
                write_vec<T, VEC>(a.dh, e, d[j], has[j] && ok0, has[j] && ok1);
                if (full && a.dz) write_vec<T, VEC>(a.dz, e, sg[j], has[j] && ok0, has[j] && ok1);
            }
    }
    if (at_row >= 0) flush();
    stage_drain(ok);
}

}  // namespace gconv
