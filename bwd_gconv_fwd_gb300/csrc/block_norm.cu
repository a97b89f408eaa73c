// block_norm.cu -- extern "C" entry points of the block norm and block join: checks,
// launch shapes, the channel-gradient finish.  The kernels are in block_norm.cuh.
#include "block_internal.h"
#include "block_stage.cuh"

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

struct FinishArgs {
    const float *part;
    int N, C, G, Cg, Z, splits;   // part: [2][splits][N][C], splits the most blocks that share rows
    int tiles, per;               // Z rows' tiles from (row / Z) tiles on were walked `per` to a block
    int next, post, gate, act;
    const void *z;
    const float *w, *s;
    float *dw2, *dw, *ds, *dzc;
};

template <typename T>
__global__ void __launch_bounds__(kFinChannels * kFinLanes) block_finish_kernel(const FinishArgs a)
{
    __shared__ float sh[2][kFinLanes][kFinChannels];
    const int cl = threadIdx.x % kFinChannels, ln = threadIdx.x / kFinChannels;
    const int c = blockIdx.x * kFinChannels + cl;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    float t2 = 0.f, tk = 0.f;
    if (c < a.C) {
        const int64_t NC = (int64_t)a.N * a.C;
        const float kc = (a.w ? a.w[c] : 1.f) * (a.s ? a.s[c] : 1.f);
        #pragma unroll 2
        for (int n = ln; n < a.N; n += kFinLanes) {
            const int64_t rb = (n * a.G + c / a.Cg) / a.Z;
            const int shares = (int)(((rb + 1) * a.tiles - 1) / a.per - rb * a.tiles / a.per) + 1;
            const float *p = a.part + (int64_t)n * a.C + c;
            float q = 0.f;
            #pragma unroll 4
            for (int i = 0; i < shares; ++i) {
                if (a.next) t2 += p[i * NC];
                if (a.post) q += p[(a.splits + i) * NC];
            }
            if (a.post && a.gate == GCONV_GATE_CHANNEL) {
                float g;
                const float dg = gate_grad(to_f(static_cast<const T *>(a.z)[(int64_t)n * a.C + c]), a.act, &g);
                if (a.dzc) a.dzc[(int64_t)n * a.C + c] = q * kc * dg;
                q *= g;
            }
            tk += q;
        }
    }
    sh[0][ln][cl] = t2;
    sh[1][ln][cl] = tk;
    __syncthreads();
    if (ln == 0 && c < a.C) {
        float u2 = 0.f, uk = 0.f;
        for (int i = 0; i < kFinLanes; ++i) { u2 += sh[0][i][cl]; uk += sh[1][i][cl]; }
        if (a.next && a.dw2) a.dw2[c] = u2;
        if (a.post && a.dw) a.dw[c] = uk * (a.s ? a.s[c] : 1.f);
        if (a.post && a.ds) a.ds[c] = uk * (a.w ? a.w[c] : 1.f);
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

// Launch shape of the staged kernels: 16 elements a thread, at most `most` threads, as many lanes
// a channel as that leaves.
bool stage_shape(const gconv_block &b, gconv_dtype dt, bool bwd, int tensors, int most, BlockShape *s)
{
    const int P = b.H * b.W, Cg = b.C / b.groups, rows = b.N * b.groups;
    const int es = dt == GCONV_BF16 ? 2 : 4;
    int vec = 16 / es;
    while (P % vec) vec >>= 1;
    const int held = vec > 1 ? vec : 2;   // positions a lane holds
    int TY = (Cg + stage_nch(vec) - 1) / stage_nch(vec);
    s->vec = vec;
    s->flat = P <= 64;
    int TX = s->flat ? pow2_up((P + held - 1) / held) : 32;
    while (TX > 1 && TX * TY > most) { TX >>= 1; s->flat = s->flat && held * TX >= P; }
    if (TX * TY > most || (!s->flat && held * TX * es < 16)) return false;
    // whole warps a row, or a power of two of rows a warp
    if (TX * TY >= 32) TY = (TY + 32 / TX - 1) / (32 / TX) * (32 / TX);
    else TY = pow2_up(TY);
    int Z = 1;
    while (TX * TY * Z < 32 || (TX * TY * Z * 2 <= most && Z < rows)) Z *= 2;
    s->PT = held * TX;
    const size_t limit = kBlockSmem;
    const int sums = bwd ? 2 : 1;
    while (true) {
        if (s->flat) {
            s->pitch = P * es;
            s->tensor = ((Z * Cg * P * es + 15 + 16 + held * TX * es) & ~15);
        } else {
            const bool aligned = (int64_t)P * es % 16 == 0 && s->PT * es % 16 == 0;
            s->pieces = (s->PT * es + 15) / 16 + (aligned ? 0 : 1);
            s->pitch = s->pieces * 16;
            s->tensor = Z * Cg * s->pitch + 16;
        }
        s->smem = (size_t)2 * tensors * s->tensor + (TX * TY > 32 ? (size_t)Z * (TX * TY / 32 + 1) * TX * stage_pairs(vec) * sums * 8 : 0);
        if (s->smem <= limit) break;
        if (Z > 1 && TX * TY * Z >= 64) Z /= 2;
        else return false;
    }
    s->lanes2 = pow2_up(s->pieces);
    s->staged = 1;
    s->TX = TX; s->TY = TY; s->Z = Z; 
    s->threads = TX * TY * Z;
    s->tiles = s->flat ? 1 : (P + s->PT - 1) / s->PT;
    s->total = (rows + Z - 1) / Z * s->tiles;
    const int per_sm = (int)std::max<size_t>(1, std::min<size_t>(kBlockSmem / (s->smem + 1024), 1024 / s->threads));
    s->per = (s->total + num_sms() * per_sm - 1) / (num_sms() * per_sm);
    s->grid = (unsigned)((s->total + s->per - 1) / s->per);
    s->splits = (s->tiles + s->per - 1) / s->per + 1;   // blocks that may share a row
    return true;
}

// Launch shape.  The widest vector of at most four positions that divides the plane (rows are
// then aligned for it);
// TX such that a channel's positions in a block are 64 bytes or more where 512 threads
// allow it.
void block_shape(const gconv_block &b, gconv_dtype dt, bool bwd, int kind, BlockShape *s)
{
    *s = BlockShape{};
    const int tensors = bwd ? (kind == kBlockJoinNext ? 5 : 3) : (kind == kBlockNorm ? 1 : 3);
    if (stage_shape(b, dt, bwd, tensors, 512, s)) return;
    *s = BlockShape{};
    const int P = b.H * b.W, Cg = b.C / b.groups, rows = b.N * b.groups;
    const int esize = dt == GCONV_BF16 ? 2 : 4;
    int vec = 4;
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
        TY = 512 / TX;
    }
    // a row's threads: whole warps, or a power of two of them in one warp
    if (TX * TY >= 32) TY = (TY + 32 / TX - 1) / (32 / TX) * (32 / TX);
    else TY = pow2_up(TY);
    int Z = 1;
    while (TX * TY * Z < 32 || (TX * TY * Z < 256 && Z * 2 <= rows && TX * TY * Z * 2 <= 256)) Z *= 2;
    s->vec = vec; s->one = one; s->TX = TX; s->TY = TY; s->Z = Z; s->PV = PV;
    s->threads = TX * TY * Z;
    s->tiles = (PV + TX - 1) / TX;
    s->per = 1;
    const int64_t row_blocks = (rows + Z - 1) / Z;
    s->splits = s->tiles;
    if (bwd && one) {
        const int64_t want = (int64_t)num_sms() * (2048 / s->threads);
        s->splits = (int)std::max<int64_t>(1, std::min<int64_t>(s->tiles, want / std::max<int64_t>(1, row_blocks)));
        const int per = (s->tiles + s->splits - 1) / s->splits;
        s->splits = (s->tiles + per - 1) / per;
    }
    s->grid = (unsigned)(row_blocks * (bwd ? s->splits : s->tiles));
    const int sums = bwd ? 2 : 1;
    s->smem = TY > 1 ? (size_t)Z * (TY + column_shares(TY)) * TX * vec * sums * sizeof(float) : 0;
}

void block_args(const gconv_block &b, gconv_dtype dt, const BlockShape &s, BlockArgs *a)
{
    a->G = b.groups; a->Cg = b.C / b.groups; a->rows = b.N * b.groups;
    a->P = b.H * b.W; a->PV = s.PV;
    a->TX = s.TX; a->TY = s.TY; a->Z = s.Z; a->tiles = s.tiles; a->splits = s.splits;
    a->PT = s.PT; a->flat = s.flat; a->per = s.per; a->total = s.total; 
    a->pitch = s.pitch; a->tensor = s.tensor; a->pieces = s.pieces; a->lanes2 = s.lanes2;
    a->bytes = (int64_t)b.N * b.C * a->P * (dt == GCONV_BF16 ? 2 : 4);
    a->whole = a->bytes % 16 == 0;
    a->eps = b.eps; a->inv_cg = 1.f / (float)a->Cg;
    cudaGetLastError();   // clear a stale error: the check after the launches is about this call
}

size_t block_ws(const gconv_block &b, gconv_dtype dt)
{
    if (b.N == 0) return 0;
    size_t most = 0;   // over the backward calls this record may be used with
    for (int kind : {kBlockNorm, kBlockJoin, kBlockJoinNext}) {
        BlockShape s;
        block_shape(b, dt, true, kind, &s);
        most = std::max(most, (size_t)2 * s.splits * b.N * b.C * sizeof(float));
    }
    return most;
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
    block_shape(*block, dtype, false, kBlockNorm, &s);
    BlockArgs a{};
    block_args(*block, dtype, s, &a);
    a.x = x; a.w2 = weight; a.next = y;
    (dtype == GCONV_BF16 ? block_fwd_bf16 : block_fwd_f32)(kBlockNorm, s, a, static_cast<cudaStream_t>(stream));
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
    const int kind = next ? kBlockJoinNext : kBlockJoin;
    block_shape(*block, dtype, false, kind, &s);
    BlockArgs a{};
    block_args(*block, dtype, s, &a);
    a.gate = block->gate; a.act = block->act;
    a.x = res; a.h = h; a.z = gate; a.w = weight; a.s = scale; a.w2 = next_weight; a.out = out; a.next = next;
    (dtype == GCONV_BF16 ? block_fwd_bf16 : block_fwd_f32)(kind, s, a, static_cast<cudaStream_t>(stream));
    return done();
}

static gconv_status finish(const gconv_block &b, gconv_dtype dt, const BlockShape &s, const BlockArgs &a, int next, int post,
                           float *dw2, float *dw, float *ds, float *dzc, cudaStream_t st)
{
    FinishArgs f{};
    f.part = a.part; f.N = b.N; f.C = b.C; f.G = b.groups; f.Cg = a.Cg; f.Z = a.Z; f.splits = s.splits;
    f.tiles = s.staged ? s.tiles : s.splits;
    f.per = s.per;
    f.next = next; f.post = post; f.gate = a.gate; f.act = a.act; f.z = a.z; f.w = a.w; f.s = a.s;
    f.dw2 = dw2; f.dw = dw; f.ds = ds; f.dzc = dzc;
    const unsigned grid = (unsigned)((b.C + kFinChannels - 1) / kFinChannels);
    if (dt == GCONV_BF16) launch_dependent(block_finish_kernel<__nv_bfloat16>, grid, kFinChannels * kFinLanes, 0, st, f);
    else launch_dependent(block_finish_kernel<float>, grid, kFinChannels * kFinLanes, 0, st, f);
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
    block_shape(*block, dtype, true, kBlockNorm, &s);
    BlockArgs a{};
    block_args(*block, dtype, s, &a);
    a.x = x; a.w2 = weight; a.dnext = dy; a.dout = dres; a.dx = dx;
    a.part = static_cast<float *>(workspace);
    (dtype == GCONV_BF16 ? block_bwd_bf16 : block_bwd_f32)(kBlockNorm, s, a, st);
    if (!dweight) return done();
    return finish(*block, dtype, s, a, 1, 0, dweight, nullptr, nullptr, nullptr, st);
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
    const int kind = dnext ? kBlockJoinNext : kBlockJoin;
    block_shape(*block, dtype, true, kind, &s);
    BlockArgs a{};
    block_args(*block, dtype, s, &a);
    a.gate = block->gate; a.act = block->act;
    a.x = out; a.h = h; a.z = gate; a.w = weight; a.s = scale; a.w2 = next_weight;
    a.dout = dout; a.dnext = dnext; a.dx = dres; a.dh = dh;
    a.dz = block->gate == GCONV_GATE_FULL ? dgate : nullptr;
    a.part = static_cast<float *>(workspace);
    (dtype == GCONV_BF16 ? block_bwd_bf16 : block_bwd_f32)(kind, s, a, st);
    float *dzc = block->gate == GCONV_GATE_CHANNEL ? static_cast<float *>(dgate) : nullptr;
    if (!dweight && !dscale && !dnext_weight && !dzc) return done();
    return finish(*block, dtype, s, a, dnext != nullptr, 1, dnext_weight, dweight, dscale, dzc, st);
}

}  // extern "C"
