// block_norm.cu -- extern "C" entry points of the block norm and block join: checks,
// launch shapes, the channel-gradient finish.  The kernels are in block_row.cuh, block_stage.cuh and
// block_norm.cuh.
#include "block_internal.h"
#include "block_row.cuh"
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
// few, so the reads' latency, not their bytes, is what the launch costs (3 to 5 us).
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
        // walkers that share the rows of image n and this channel's group
        const int g = c / a.Cg;
        auto shares = [&](int n) {
            const int at = (n * a.G + g) / a.Z * a.tiles;
            return (at + a.tiles - 1) / a.per - at / a.per + 1;
        };
        const float *p = a.part + c;
        if (a.post && a.gate == GCONV_GATE_CHANNEL) {
            for (int n = ln; n < a.N; n += kFinLanes) {
                const int m = shares(n);
                float q = 0.f;
                #pragma unroll 4
                for (int i = 0; i < m; ++i) {
                    if (a.next) t2 += p[i * NC + (int64_t)n * a.C];
                    q += p[(a.splits + i) * NC + (int64_t)n * a.C];
                }
                float v;
                const float dv = gate_grad(to_f(static_cast<const T *>(a.z)[(int64_t)n * a.C + c]), a.act, &v);
                if (a.dzc) a.dzc[(int64_t)n * a.C + c] = q * kc * dv;
                tk = fmaf(q, v, tk);
            }
        } else {
            // images and walkers as one sum, so that its terms are all in flight
            #pragma unroll 8
            for (int i = ln; i < a.N * a.splits; i += kFinLanes) {
                const int n = i / a.splits, m = i - n * a.splits;
                if (m < shares(n)) {
                    const int64_t at = (int64_t)n * a.C + m * NC;
                    if (a.next) t2 += p[at];
                    if (a.post) tk += p[at + a.splits * NC];
                }
            }
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

// Launch shape of the staged kernels: as many lanes a channel as the elements a thread holds and
// shared memory leave.  Two tiles stand in shared memory, a channel's positions in one being 64
// bytes, else 32, in one block, else with the channels over a cluster of two; then one tile in a
// cluster of two; then larger clusters.  Measured: norm of [42,728,28,28] bf16, one block and 16
// bytes 56 us, two blocks and 32 bytes 41, four and 64 bytes 61; join backward of [32,1024,7,7]
// fp32, one tile in two blocks 29 us, two tiles in four 38, in eight 68: a cluster's barrier costs
// more than copies that wait, and both less than sectors read twice.  The tensors are counted as if the
// call had a full gate and every gradient: without them their shared memory stands empty.
bool stage_shape(const gconv_block &b, gconv_dtype dt, bool bwd, int kind, BlockShape *s)
{
    const int tensors = bwd ? (kind == kBlockJoinNext ? 5 : 3) : (kind == kBlockNorm ? 1 : 3), sums = bwd ? 2 : 1;
    const int P = b.H * b.W, Cg = b.C / b.groups, rows = b.N * b.groups;
    const int es = dt == GCONV_BF16 ? 2 : 4;
    int vec = 16 / es;
    while (P % vec) vec >>= 1;
    // threads of a block, and those an SM's registers hold: one block in the gradient of a join, else two
    const int most = stage_threads(vec), resident = bwd && kind != kBlockNorm ? most : 2 * most;
    const int held = vec > 1 ? vec : 2;   // positions a lane holds
    const int widest = P <= 64 ? pow2_up((P + held - 1) / held) : 32;

    auto fits = [&](int cluster, int TX, int Z, int stages, int least, int nch) {
        const int Cc = (Cg + cluster - 1) / cluster, share = (Cc + nch - 1) / nch;
        if ((cluster - 1) * Cc >= Cg) return false;            // a block without channels
        // whole warps a row, or a power of two of rows a warp
        const int TY = TX * share >= 32 || cluster > 1 ? (share + 32 / TX - 1) / (32 / TX) * (32 / TX) : pow2_up(share);
        if (TX * TY * Z > most) return false;
        s->flat = P <= 64 && held * TX >= P;
        s->PT = held * TX;
        if (!s->flat && s->PT * es < least) return false;
        s->boxes = s->box_rows = s->pieces = 0;
        const bool aligned = (int64_t)P * es % 16 == 0 && s->PT * es % 16 == 0;
        if (s->flat) {
            s->pitch = P * es;
            s->tensor = Z * Cc * P * es + 16 + 16 + held * TX * es;
        } else if (aligned && s->PT * es >= 64) {
            s->pitch = s->PT * es;
            s->boxes = (Z * Cc + 255) / 256;
            s->box_rows = ((Z * Cc + s->boxes - 1) / s->boxes + 1) & ~1;   // 128 bytes or a multiple: the next box follows
            s->tensor = s->boxes * s->box_rows * s->pitch;
        } else {
            s->pieces = (s->PT * es + 15) / 16 + (aligned ? 0 : 1);
            s->pitch = s->pieces * 16;
            s->tensor = Z * Cc * s->pitch + 16;
        }
        s->tensor = (s->tensor + kStageZeros + 127) & ~127;
        const size_t width = (size_t)TX * stage_pairs(vec) * sums * 8;   // of column_roots
        s->smem = 128 + (size_t)stages * tensors * s->tensor;
        if (TX * TY > 32 || cluster > 1) s->smem += 2 * (Z * (TX * TY / 32) + (cluster > 1 ? cluster : 0)) * width;
        if (s->smem > kBlockSmem) return false;
        s->TX = TX; s->TY = TY; s->Z = Z; s->stages = stages; s->cluster = cluster; s->Cc = Cc;
        s->threads = TX * TY * Z;
        return true;
    };
    bool found = false;
    // stages, blocks of a cluster, least bytes of a channel
    const int tries[][3] = {{2, 1, 64}, {2, 1, 32}, {2, 2, 64}, {2, 2, 32}, {1, 2, 32}, {2, 4, 32}, {1, 4, 32}, {2, 8, 32}, {1, 8, 16}};
    int nch = stage_nch(vec);
    for (const auto &k : tries)
        for (int TX = widest; TX >= 1 && !found; TX >>= 1) {
            int Z = 1;
            while (k[1] == 1 && TX * pow2_up((Cg + nch - 1) / nch) * Z < 32) Z *= 2;
            found = fits(k[1], TX, Z, k[0], k[2], nch);
        }
    if (!found) return false;
    // several rows a block where one gives it few threads
    while (s->cluster == 1 && s->threads * 2 <= most / 2 && s->Z < rows) {
        const BlockShape kept = *s;
        if (!fits(1, kept.TX, kept.Z * 2, kept.stages, 16, nch)) { *s = kept; break; }
    }
    // fewer channels a thread where shared memory leaves the SM's threads unused: a tile's chain of
    // instructions is then shorter
    auto blocks_an_sm = [&] {
        return (int)std::max<size_t>(1, std::min<size_t>(kBlockSmem / (s->smem + 1024), resident / s->threads));
    };
    while (nch > 1 && s->TX * s->TY >= 32 && 2 * s->threads * blocks_an_sm() <= resident) {
        const BlockShape kept = *s;
        if (!fits(kept.cluster, kept.TX, kept.Z, kept.stages, 16, nch / 2)) { *s = kept; break; }
        nch /= 2;
    }
    s->vec = vec;
    s->staged = 1;
    s->tiles = s->flat ? 1 : (P + s->PT - 1) / s->PT;
    s->total = (rows + s->Z - 1) / s->Z * s->tiles;
    const int per_sm = blocks_an_sm();
    const int walkers = std::max(1, num_sms() * per_sm / s->cluster);
    s->per = (s->total + walkers - 1) / walkers;
    s->grid = (unsigned)((s->total + s->per - 1) / s->per) * s->cluster;
    s->splits = (s->tiles + s->per - 1) / s->per + 1;   // walkers that may share a row
    return true;
}

// Launch shape of the row kernels: a lane a vector up to a warp, then as many channels a lane as it
// holds, and fewer again, and fewer rows a block, while there are more SMs than work.  The gradients'
// blocks are as many as the SMs hold at once, so that channel sums are put down once.
bool row_shape(const gconv_block &b, gconv_dtype dt, bool bwd, int kind, BlockShape *s)
{
    const int es = dt == GCONV_BF16 ? 2 : 4, Cg = b.C / b.groups, rows = b.N * b.groups;
    if (b.H * b.W != 1) return false;
    if (bwd && b.groups > 1 && Cg * es < 32) return false;   // a block's rows are a group's: shorter than a sector
    const int vec = Cg % (16 / es) ? 1 : 16 / es, vectors = Cg / vec;
    // twice as many channels a thread where a row is too long, and where there is little to hold: norm of
    // [65536,1024] bf16 69 us with 8 a thread, 59 with 16; gradient of a join 465 and 508
    s->held = vec > 1 && (Cg > kRowThreads * kRowHeld || (vec == 8 && !bwd && kind == kBlockNorm)) ? 2 * kRowHeld : kRowHeld;
    const int nv = s->held / vec;
    if (vectors > kRowThreads * nv) return false;
    const int walked = bwd ? b.N : rows, groups = bwd ? b.groups : 1;   // rows a walker may have, kinds of walkers
    s->TY = std::min(pow2_up(vectors), std::max(32, pow2_up((vectors + nv - 1) / nv)));
    while (s->TY < kRowThreads && s->TY < vectors && (int64_t)rows * s->TY < num_sms() * 256) s->TY *= 2;
    s->threads = std::max(256, s->TY);
    s->Z = s->threads / s->TY;
    while (s->Z > 1 && s->threads > 32 && (int64_t)((walked + s->Z - 1) / s->Z) * groups < num_sms()) {
        s->Z /= 2;
        s->threads /= 2;
    }
    const int threads = !bwd ? 2048 : kind == kBlockNorm && s->held == kRowHeld ? 1024 : 512;   // of an SM, by its registers
    const int blocks = (walked + s->Z - 1) / s->Z, room = num_sms() * threads / s->threads;
    s->splits = std::min(blocks, std::max(1, room / groups));
    s->grid = (unsigned)(s->splits * groups);
    s->images = 1;
    s->row = 1;
    s->vec = vec;
    s->TX = s->tiles = s->per = s->cluster = 1;
    s->smem = bwd && s->Z > 1 ? (size_t)s->threads * nv * vec * sizeof(float) : 0;
    return true;
}

// Launch shape of a call; of the walking kernels where the staged ones do not fit: 32 positions of
// a row a block.
void block_shape(const gconv_block &b, gconv_dtype dt, bool bwd, int kind, BlockShape *s)
{
    *s = BlockShape{};
    if (row_shape(b, dt, bwd, kind, s)) return;
    s->images = b.N;
    if (stage_shape(b, dt, bwd, kind, s)) return;
    *s = BlockShape{};
    s->images = b.N;
    const int P = b.H * b.W, rows = b.N * b.groups;
    // half as many where the SMs would not all have a block, but 32 bytes
    s->TX = std::min(32, pow2_up(P));
    while (s->TX * (dt == GCONV_BF16 ? 2 : 4) > 32 && rows * ((P + s->TX - 1) / s->TX) < num_sms()) s->TX /= 2;
    s->TY = 512 / s->TX;
    s->Z = 1;
    s->cluster = 1;
    s->threads = s->TX * s->TY;
    s->tiles = s->splits = (P + s->TX - 1) / s->TX;
    s->per = 1;
    s->grid = (unsigned)(rows * s->tiles);
    s->smem = (size_t)(s->TY + column_shares(s->TY)) * s->TX * (bwd ? 2 : 1) * sizeof(float);
}

void block_args(const gconv_block &b, gconv_dtype dt, const BlockShape &s, BlockArgs *a)
{
    a->G = b.groups; a->Cg = b.C / b.groups; a->rows = b.N * b.groups;
    a->P = b.H * b.W;
    a->TX = s.TX; a->TY = s.TY; a->Z = s.Z; a->tiles = s.tiles; a->splits = s.splits;
    a->PT = s.PT; a->flat = s.flat; a->per = s.per; a->total = s.total; a->stages = s.stages; a->cluster = s.cluster; a->Cc = s.Cc;
    a->pitch = s.pitch; a->tensor = s.tensor; a->boxes = s.boxes; a->box_rows = s.box_rows;
    a->box_bytes = s.box_rows * s.pitch;
    a->pieces = s.pieces;
    a->err = device_error_word();
    a->wait_ns = (uint64_t)wait_limit();
    a->bytes = (int64_t)b.N * b.C * a->P * (dt == GCONV_BF16 ? 2 : 4);
    a->eps = b.eps; a->inv_cg = 1.f / (float)a->Cg;
    cudaGetLastError();   // clear a stale error: the check after the launches is about this call
}

// Launches the forward or backward kernel: the tensors' maps are in the order the kernels stage them.
gconv_status run_block(bool bwd, int kind, const gconv_block &b, gconv_dtype dt, const BlockShape &s, const BlockArgs &a,
                       cudaStream_t st)
{
    const bool next = kind != kBlockJoin, post = kind != kBlockNorm;
    const void *src[5] = {bwd ? a.dout : a.x};
    int n = 1;
    if (bwd && next) { src[n++] = a.x; src[n++] = a.dnext; }
    if (post) { src[n++] = a.h; src[n++] = a.gate == GCONV_GATE_FULL ? a.z : nullptr; }
    if (!a.err) return GCONV_ERR_CUDA;
    StageMaps maps;
    for (int i = 0; s.boxes > 0 && i < n; ++i)
        if (src[i] && !encode_matrix_tmap(&maps.m[i], dt, src[i], (uint64_t)a.P, (uint64_t)b.N * b.C, (uint32_t)s.PT,
                                          (uint32_t)s.box_rows))
            return GCONV_ERR_CUDA;
    if (bwd) (dt == GCONV_BF16 ? block_bwd_bf16 : block_bwd_f32)(kind, s, a, maps, st);
    else (dt == GCONV_BF16 ? block_fwd_bf16 : block_fwd_f32)(kind, s, a, maps, st);
    return cudaGetLastError() == cudaSuccess ? GCONV_OK : GCONV_ERR_CUDA;
}

size_t block_ws(const gconv_block &b, gconv_dtype dt)
{
    if (b.N == 0) return 0;
    size_t most = 0;   // over the backward calls this record may be used with
    for (int kind : {kBlockNorm, kBlockJoin, kBlockJoinNext}) {
        BlockShape s;
        block_shape(b, dt, true, kind, &s);
        most = std::max(most, (size_t)2 * s.splits * s.images * b.C * sizeof(float));
    }
    return most;
}

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
    return run_block(false, kBlockNorm, *block, dtype, s, a, static_cast<cudaStream_t>(stream));
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
    return run_block(false, kind, *block, dtype, s, a, static_cast<cudaStream_t>(stream));
}

static gconv_status finish(const gconv_block &b, gconv_dtype dt, const BlockShape &s, const BlockArgs &a, int next, int post,
                           float *dw2, float *dw, float *ds, float *dzc, cudaStream_t st)
{
    FinishArgs f{};
    f.part = a.part; f.N = s.images; f.C = b.C; f.G = b.groups; f.Cg = a.Cg; f.Z = a.Z; f.splits = s.splits;
    f.tiles = s.staged ? s.tiles : s.splits;
    f.per = s.per;
    if (s.row) f.Z = b.groups;   // every walker has a share of the one row of sums
    f.next = next; f.post = post; f.gate = s.row && a.gate == GCONV_GATE_CHANNEL ? GCONV_GATE_FULL : a.gate; f.act = a.act; f.z = a.z; f.w = a.w; f.s = a.s;
    f.dw2 = dw2; f.dw = dw; f.ds = ds; f.dzc = dzc;
    const unsigned grid = (unsigned)((b.C + kFinChannels - 1) / kFinChannels);
    if (dt == GCONV_BF16) launch_dependent(block_finish_kernel<__nv_bfloat16>, grid, kFinChannels * kFinLanes, 0, st, f);
    else launch_dependent(block_finish_kernel<float>, grid, kFinChannels * kFinLanes, 0, st, f);
    return cudaGetLastError() == cudaSuccess ? GCONV_OK : GCONV_ERR_CUDA;
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
    BlockShape s;
    block_shape(*block, dtype, true, kBlockNorm, &s);
    if (!workspace || workspace_bytes < block_ws(*block, dtype)) return GCONV_ERR_WORKSPACE;
    BlockArgs a{};
    block_args(*block, dtype, s, &a);
    a.x = x; a.w2 = weight; a.dnext = dy; a.dout = dres; a.dx = dx;
    a.part = static_cast<float *>(workspace);
    const gconv_status r = run_block(true, kBlockNorm, *block, dtype, s, a, st);
    if (r != GCONV_OK || !dweight) return r;
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
    BlockShape s;
    const int kind = dnext ? kBlockJoinNext : kBlockJoin;
    block_shape(*block, dtype, true, kind, &s);
    if (!workspace || workspace_bytes < block_ws(*block, dtype)) return GCONV_ERR_WORKSPACE;
    BlockArgs a{};
    block_args(*block, dtype, s, &a);
    a.gate = block->gate; a.act = block->act;
    a.x = out; a.h = h; a.z = gate; a.w = weight; a.s = scale; a.w2 = next_weight;
    a.dout = dout; a.dnext = dnext; a.dx = dres; a.dh = dh;
    a.dz = block->gate == GCONV_GATE_FULL || s.row ? dgate : nullptr;
    a.part = static_cast<float *>(workspace);
    const gconv_status r = run_block(true, kind, *block, dtype, s, a, st);
    if (r != GCONV_OK) return r;
    float *dzc = block->gate == GCONV_GATE_CHANNEL && !s.row ? static_cast<float *>(dgate) : nullptr;
    if (!dweight && !dscale && !dnext_weight && !dzc) return GCONV_OK;
    return finish(*block, dtype, s, a, dnext != nullptr, 1, dnext_weight, dweight, dscale, dzc, st);
}

}  // extern "C"
