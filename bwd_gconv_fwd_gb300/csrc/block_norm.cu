// block_norm.cu -- extern "C" entry points of the block norm and block join: checks,
// launch shapes, the channel-gradient finish.  The kernels are in block_norm.cuh.
#include "block_internal.h"

#include <algorithm>
#include <climits>

namespace gconv {

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Channel gradients from the blocks' sums, in a fixed order: part[0] gives dw2, part[1] the
// sum q of dx * (h r) per image and channel (times the gate unless it is a channel gate), and
//   dz[n][c] = act'(z) s w q,   dk[c] = sum_n act(z) q,   dw = s dk,   ds = w dk.
// Eight channels a block, 32 threads a channel: C is at most a few thousand and the sums
// few, so the reads' latency, not their bytes, is what the launch costs.
constexpr int kFinChannels = 8, kFinLanes = 32;

template <typename T>
__global__ void __launch_bounds__(kFinChannels * kFinLanes)
block_finish_kernel(const float *part, int N, int C, int splits, int next, int post, int gate, int act, const T *zg,
                    const float *w, const float *s, float *dw2, float *dw, float *ds, float *dzc)
{
    __shared__ float sh[2][kFinLanes][kFinChannels];
    const int cl = threadIdx.x % kFinChannels, ln = threadIdx.x / kFinChannels;
    const int c = blockIdx.x * kFinChannels + cl;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    float t2 = 0.f, tk = 0.f;
    if (c < C) {
        const int64_t NC = (int64_t)N * C;
        const float *p0 = part, *p1 = part + splits * NC;
        const bool per_image = post && gate == GCONV_GATE_CHANNEL;
        const float kc = (w ? w[c] : 1.f) * (s ? s[c] : 1.f);
        if (next && dw2)
            for (int64_t i = ln; i < (int64_t)N * splits; i += kFinLanes) t2 += p0[i * C + c];   // [splits][N][C]
        if (per_image) {
            for (int n = ln; n < N; n += kFinLanes) {
                float q = 0.f;
                for (int i = 0; i < splits; ++i) q += p1[i * NC + (int64_t)n * C + c];
                float g;
                const float dg = gate_grad(to_f(zg[(int64_t)n * C + c]), act, &g);
                if (dzc) dzc[(int64_t)n * C + c] = q * kc * dg;
                tk += q * g;
            }
        } else if (post) {
            for (int64_t i = ln; i < (int64_t)N * splits; i += kFinLanes) tk += p1[i * C + c];
        }
    }
    sh[0][ln][cl] = t2;
    sh[1][ln][cl] = tk;
    __syncthreads();
    if (ln == 0 && c < C) {
        float u2 = 0.f, uk = 0.f;
        for (int i = 0; i < kFinLanes; ++i) { u2 += sh[0][i][cl]; uk += sh[1][i][cl]; }
        if (next && dw2) dw2[c] = u2;
        if (post && dw) dw[c] = uk * (s ? s[c] : 1.f);
        if (post && ds) ds[c] = uk * (w ? w[c] : 1.f);
    }
}

bool check_block(const gconv_block *b, gconv_dtype dt)
{
    if (!b || (dt != GCONV_F32 && dt != GCONV_BF16)) return false;
    if (b->N < 0 || b->C < 1 || b->H < 1 || b->W < 1 || b->groups < 1 || b->C % b->groups) return false;
    if (!(b->eps >= 0.f) || b->eps > 3e38f) return false;
    if (b->gate < GCONV_GATE_NONE || b->gate > GCONV_GATE_CHANNEL) return false;
    if (b->act < GCONV_ACT_NONE || b->act > GCONV_ACT_SILU) return false;
    const int64_t plane = (int64_t)b->H * b->W, lim = INT_MAX;
    if (plane > lim || plane * b->C > lim || plane * b->C * b->N > lim) return false;
    return true;
}

int pow2_up(int v)
{
    int p = 1;
    while (p < v) p <<= 1;
    return p;
}

// Launch shape.  The widest vector that divides the plane (rows are then aligned for it);
// TX such that a channel's positions in a block are 64 bytes or more where 512 threads
// allow it.
void block_shape(const gconv_block &b, gconv_dtype dt, bool bwd, BlockShape *s)
{
    const int P = b.H * b.W, Cg = b.C / b.groups, rows = b.N * b.groups;
    const int esize = dt == GCONV_BF16 ? 2 : 4;
    int vec = 16 / esize;
    while (P % vec) vec >>= 1;
    int nch = block_nch(vec);
    int one = 1;
    if ((Cg + nch - 1) / nch > 512) { one = 0; vec = 1; nch = block_nch(1); }
    const int PV = P / vec;
    int TX, TY;
    if (one) {
        const int ty = (Cg + nch - 1) / nch;
        TX = std::min(32, pow2_up(PV));
        while (TX > 1 && TX * ty > 512) TX >>= 1;
        while (TX > 1 && TX * ty > 256 && TX * vec * esize > 64) TX >>= 1;
        TY = ty;
    } else {
        TX = std::min(32, pow2_up(PV));
        TY = 256 / TX;
    }
    // a row's threads: whole warps, or a power of two of them in one warp
    if (TX * TY >= 32) TY = (TY + 32 / TX - 1) / (32 / TX) * (32 / TX);
    else TY = pow2_up(TY);
    int Z = 1;
    while (TX * TY * Z < 32 || (TX * TY * Z < 256 && Z * 2 <= rows && TX * TY * Z * 2 <= 256)) Z *= 2;
    s->vec = vec; s->one = one; s->TX = TX; s->TY = TY; s->Z = Z; s->PV = PV;
    s->threads = TX * TY * Z;
    s->tiles = (PV + TX - 1) / TX;
    const int64_t row_blocks = (rows + Z - 1) / Z;
    s->splits = s->tiles;
    if (bwd && one) {
        const int64_t want = (int64_t)num_sms() * (2048 / s->threads);
        s->splits = (int)std::max<int64_t>(1, std::min<int64_t>(s->tiles, want / std::max<int64_t>(1, row_blocks)));
        const int per = (s->tiles + s->splits - 1) / s->splits;
        s->splits = (s->tiles + per - 1) / per;
    }
    s->grid = (unsigned)(row_blocks * (bwd ? s->splits : s->tiles));
    const int per_row = TX * TY;
    s->smem = per_row > 32 ? (size_t)Z * (per_row / 32 + 1) * TX * vec * (bwd ? 2 : 1) * sizeof(float) : 0;
}

void block_args(const gconv_block &b, const BlockShape &s, BlockArgs *a)
{
    a->G = b.groups; a->Cg = b.C / b.groups; a->rows = b.N * b.groups;
    a->P = b.H * b.W; a->PV = s.PV;
    a->TX = s.TX; a->TY = s.TY; a->Z = s.Z; a->tiles = s.tiles; a->splits = s.splits;
    a->eps = b.eps; a->inv_cg = 1.f / (float)a->Cg;
    cudaGetLastError();   // clear a stale error: the check after the launches is about this call
}

size_t block_ws(const gconv_block &b, gconv_dtype dt)
{
    if (b.N == 0) return 0;
    BlockShape s;
    block_shape(b, dt, true, &s);
    return (size_t)2 * s.splits * b.N * b.C * sizeof(float);
}

gconv_status done() { return cudaGetLastError() == cudaSuccess ? GCONV_OK : GCONV_ERR_CUDA; }

// dw2, dw, ds, dz of an empty batch: sums over no terms
gconv_status zero(float *p, int n, cudaStream_t st)
{
    if (p && cudaMemsetAsync(p, 0, (size_t)n * sizeof(float), st) != cudaSuccess) return GCONV_ERR_CUDA;
    return GCONV_OK;
}

}  // namespace

}  // namespace gconv

using namespace gconv;

extern "C" {

size_t gconv_block_workspace_size(const gconv_block *block, gconv_dtype dtype)
{
    return check_block(block, dtype) ? block_ws(*block, dtype) : (size_t)-1;
}

gconv_status gconv_norm_fwd(const gconv_block *block, gconv_dtype dtype, const void *x, const float *weight, void *y,
                            void *stream)
{
    if (!check_block(block, dtype)) return GCONV_ERR_INVALID_ARG;
    if (block->N == 0) return GCONV_OK;
    if (!x || !y || !aligned16(x) || !aligned16(y) || !aligned16(weight)) return GCONV_ERR_INVALID_ARG;
    BlockShape s;
    block_shape(*block, dtype, false, &s);
    BlockArgs a{};
    block_args(*block, s, &a);
    a.x = x; a.w2 = weight; a.next = y;
    block_fwd_launch(kBlockNorm, dtype, s, a, static_cast<cudaStream_t>(stream));
    return done();
}

gconv_status gconv_join_fwd(const gconv_block *block, gconv_dtype dtype, const void *res, const void *h,
                            const void *gate, const float *weight, const float *scale, const float *next_weight,
                            void *out, void *next, void *stream)
{
    if (!check_block(block, dtype)) return GCONV_ERR_INVALID_ARG;
    if (block->N == 0) return GCONV_OK;
    const bool gated = block->gate != GCONV_GATE_NONE;
    if (!res || !h || !out || gated != (gate != nullptr) || (next_weight && !next)) return GCONV_ERR_INVALID_ARG;
    for (const void *p : {res, h, gate, (const void *)weight, (const void *)scale, (const void *)next_weight,
                          (const void *)out, (const void *)next})
        if (!aligned16(p)) return GCONV_ERR_INVALID_ARG;
    BlockShape s;
    block_shape(*block, dtype, false, &s);
    BlockArgs a{};
    block_args(*block, s, &a);
    a.gate = block->gate; a.act = block->act;
    a.x = res; a.h = h; a.z = gate; a.w = weight; a.s = scale; a.w2 = next_weight; a.out = out; a.next = next;
    block_fwd_launch(next ? kBlockJoinNext : kBlockJoin, dtype, s, a, static_cast<cudaStream_t>(stream));
    return done();
}

static gconv_status finish(const gconv_block &b, gconv_dtype dt, const BlockArgs &a, int next, int post, float *dw2,
                           float *dw, float *ds, float *dzc, cudaStream_t st)
{
    const unsigned grid = (unsigned)((b.C + kFinChannels - 1) / kFinChannels);
    const int threads = kFinChannels * kFinLanes;
    if (dt == GCONV_BF16)
        launch_dependent(block_finish_kernel<__nv_bfloat16>, grid, threads, 0, st, (const float *)a.part, b.N, b.C,
                         a.splits, next, post, a.gate, a.act, static_cast<const __nv_bfloat16 *>(a.z), a.w, a.s, dw2,
                         dw, ds, dzc);
    else
        launch_dependent(block_finish_kernel<float>, grid, threads, 0, st, (const float *)a.part, b.N, b.C, a.splits,
                         next, post, a.gate, a.act, static_cast<const float *>(a.z), a.w, a.s, dw2, dw, ds, dzc);
    return done();
}

gconv_status gconv_norm_bwd(const gconv_block *block, gconv_dtype dtype, const void *x, const float *weight,
                            const void *dy, const void *dres, void *dx, float *dweight, void *workspace,
                            size_t workspace_bytes, void *stream)
{
    if (!check_block(block, dtype)) return GCONV_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (block->N == 0) return zero(dweight, block->C, st);
    if (!x || !dy || !dx) return GCONV_ERR_INVALID_ARG;
    for (const void *p : {x, (const void *)weight, dy, dres, (const void *)dx, (const void *)dweight,
                          (const void *)workspace})
        if (!aligned16(p)) return GCONV_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < block_ws(*block, dtype)) return GCONV_ERR_WORKSPACE;
    BlockShape s;
    block_shape(*block, dtype, true, &s);
    BlockArgs a{};
    block_args(*block, s, &a);
    a.x = x; a.w2 = weight; a.dnext = dy; a.dout = dres; a.dx = dx;
    a.part = static_cast<float *>(workspace);
    block_bwd_launch(kBlockNorm, dtype, s, a, st);
    if (!dweight) return done();
    return finish(*block, dtype, a, 1, 0, dweight, nullptr, nullptr, nullptr, st);
}

gconv_status gconv_join_bwd(const gconv_block *block, gconv_dtype dtype, const void *out, const void *h,
                            const void *gate, const float *weight, const float *scale, const float *next_weight,
                            const void *dout, const void *dnext, void *dres, void *dh, void *dgate, float *dweight,
                            float *dscale, float *dnext_weight, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!check_block(block, dtype)) return GCONV_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (block->N == 0) {
        if (zero(dweight, block->C, st) != GCONV_OK || zero(dscale, block->C, st) != GCONV_OK) return GCONV_ERR_CUDA;
        return dnext ? zero(dnext_weight, block->C, st) : GCONV_OK;
    }
    const bool gated = block->gate != GCONV_GATE_NONE;
    if (!h || !dh || gated != (gate != nullptr) || (!gated && dgate)) return GCONV_ERR_INVALID_ARG;
    if (dnext ? !out || !dres : !dout || dres || dnext_weight || next_weight) return GCONV_ERR_INVALID_ARG;
    for (const void *p : {out, h, gate, (const void *)weight, (const void *)scale, (const void *)next_weight, dout, dnext,
                          (const void *)dres, (const void *)dh, (const void *)dgate, (const void *)dweight,
                          (const void *)dscale, (const void *)dnext_weight, (const void *)workspace})
        if (!aligned16(p)) return GCONV_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < block_ws(*block, dtype)) return GCONV_ERR_WORKSPACE;
    BlockShape s;
    block_shape(*block, dtype, true, &s);
    BlockArgs a{};
    block_args(*block, s, &a);
    a.gate = block->gate; a.act = block->act;
    a.x = out; a.h = h; a.z = gate; a.w = weight; a.s = scale; a.w2 = next_weight;
    a.dout = dout; a.dnext = dnext; a.dx = dres; a.dh = dh;
    a.dz = block->gate == GCONV_GATE_FULL ? dgate : nullptr;
    a.part = static_cast<float *>(workspace);
    block_bwd_launch(dnext ? kBlockJoinNext : kBlockJoin, dtype, s, a, st);
    float *dzc = block->gate == GCONV_GATE_CHANNEL ? static_cast<float *>(dgate) : nullptr;
    if (!dweight && !dscale && !dnext_weight && !dzc) return done();
    return finish(*block, dtype, a, dnext != nullptr, 1, dnext_weight, dweight, dscale, dzc, st);
}

}  // extern "C"
