// CPU replay of the selective scan's launch plans (scan.cu, plan_scan) over random sizes: the pieces cover every tile once, the blocks
// every channel, shared memory and grids stay within the device's, and the workspace's parts lie one after the other.
// Usage: scan_plan_replay <seed> <count>
#include "../../bwd_gconv_fwd_gb300/csrc/scan.cu"
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>
namespace gconv {
int num_sms() { return 152; }
void scan_fwd_bf16(const ScanShape &, bool, const ScanArgs &, cudaStream_t) {}
void scan_fwd_f32(const ScanShape &, bool, const ScanArgs &, cudaStream_t) {}
void scan_bwd_bf16(const ScanShape &, bool, const ScanArgs &, cudaStream_t) {}
void scan_bwd_f32(const ScanShape &, bool, const ScanArgs &, cudaStream_t) {}
}
static long errors = 0, plans = 0, cuts = 0, pairs = 0;
#define CHECK(cond, what) do { if (!(cond)) { if (errors++ < 10) printf("FAIL: %s: N %d C %d L %d groups %d states %d back %d\n", what, \
    s.N, s.C, s.L, s.groups, s.states, back); } } while (0)

static void look(const gconv_scan &s, bool back)
{
    ScanPlan p;
    if (!plan_scan(s, back, &p)) return;
    ++plans;
    const int Cg = s.C / s.groups, S = s.states;
    if (p.token) {
        CHECK(!back && s.L <= kTokenMost && p.ncb * 32 >= Cg && (p.ncb - 1) * 32 < Cg && p.bytes == 0, "short form");
        CHECK((int64_t)p.shape.grid == (int64_t)((s.N + p.token - 1) / p.token) * s.groups * p.ncb, "short grid");
        return;
    }
    const int tiles = (s.L + kScanTile - 1) / kScanTile, per = p.shape.warps * kScanOwn * p.sets;
    cuts += p.chunks > 1;
    pairs += p.sets > 1;
    CHECK(p.shape.warps >= 1 && p.shape.warps <= 4 && p.ends.warps == p.shape.warps, "warps");
    CHECK((int64_t)p.ncb * per >= Cg && (int64_t)(p.ncb - 1) * per < Cg, "channels");
    CHECK(p.sets == 1 || (back && S <= kScanStates), "sets");
    CHECK((int64_t)p.chunks * p.chunk_tiles >= tiles && (int64_t)(p.chunks - 1) * p.chunk_tiles < tiles, "tiles");
    CHECK(p.shape.smem <= 227 * 1024 && p.ends.smem <= 227 * 1024, "shared memory");
    CHECK((int64_t)p.shape.grid == (int64_t)s.N * s.groups * p.ncb * p.chunks, "grid");
    // the workspace: each part behind the one before, on 16 bytes
    const size_t pieces = (size_t)s.N * p.chunks, f = sizeof(float);
    size_t at = 0;
    auto part = [&](size_t from, size_t n, const char *what) {
        CHECK(from % 16 == 0 && from >= at, what);
        at = from + n * f;
    };
    if (p.chunks > 1) {
        part(p.o_init, pieces * S * s.C, "init");
        part(p.o_dsum, pieces * s.C, "dsum");
    }
    if (back) {
        if (p.ncb > 1) part(p.o_part, (size_t)s.N * s.groups * p.ncb * 2 * S * s.L, "part");
        part(p.o_pA, pieces * s.C * S, "pA");
        part(p.o_pD, pieces * s.C, "pD");
        part(p.o_pb, pieces * s.C, "pb");
    }
    CHECK(at <= p.bytes, "workspace");
}

int main(int argc, char **argv)
{
    std::mt19937 rng(argc > 1 ? atoi(argv[1]) : 1);
    const int count = argc > 2 ? atoi(argv[2]) : 1000;
    auto log = [&](double lo, double hi) { return (int)std::exp(std::uniform_real_distribution<double>(std::log(lo), std::log(hi + 0.5))(rng)); };
    for (int i = 0; i < count; ++i) {
        gconv_scan s{};
        s.groups = log(1, 64);
        s.C = s.groups * log(1, 4096.0 / s.groups);
        s.N = log(1, 512);
        s.L = log(1, 1 << 20);
        s.states = log(1, 256);
        if (std::max((double)s.C, (double)s.groups * s.states) * s.L * s.N > std::ldexp(1.0, 40)) continue;
        for (gconv_dtype dt : {GCONV_F32, GCONV_BF16})
            if (!check_scan(&s, dt)) { printf("FAIL: refused\n"); ++errors; }
        look(s, false);
        look(s, true);
    }
    printf("plans: %ld cut: %ld in sets: %ld errors: %ld\n", plans, cuts, pairs, errors);
    return errors ? 1 : 0;
}
