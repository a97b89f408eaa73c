// CPU replay of the selective scan's launch plans (scan.cu, plan_scan) for as many channels as the header allows, up to 2^31 - 1: the
// blocks cover every channel, grids are positive, and the workspace has room for its parts.
// Usage: scan_wide_replay <seed> <count>
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
static long errors = 0, plans = 0, last = 0;
#define CHECK(cond, what) do { if (!(cond)) { if (errors++ < 10) printf("FAIL: %s: N %d C %d L %d groups %d states %d back %d\n", what, \
    s.N, s.C, s.L, s.groups, s.states, back); } } while (0)

static void look(const gconv_scan &s, bool back)
{
    ScanPlan p;
    const bool fits = plan_scan(s, back, &p);
    // a block has at least eight channels of a group, so that a grid passes 2^31 only with many groups
    CHECK(fits || (int64_t)s.N * s.groups > INT_MAX / 64, "refused");
    if (!fits) return;
    ++plans;
    const int64_t Cg = s.C / s.groups, per = p.token ? 32 : p.shape.warps * kScanOwn * p.sets;
    last += Cg > INT_MAX - per;
    CHECK(p.ncb >= 1 && p.ncb * per >= Cg && (p.ncb - 1) * per < Cg, "channels");
    const int64_t items = p.token ? (s.N + p.token - 1) / p.token : (int64_t)s.N * p.chunks;
    CHECK((int64_t)p.shape.grid == items * s.groups * p.ncb && p.shape.grid <= INT_MAX, "grid");
    if (p.token) return;
    const int64_t one = p.shape.warps * kScanOwn;
    CHECK((int64_t)p.ends.grid == items * s.groups * (back ? (Cg - 1) / one + 1 : p.ncb) && p.ends.grid <= INT_MAX, "first pass");
    if (back) CHECK(p.bytes >= (size_t)items * s.C * (s.states + 2) * sizeof(float), "workspace");
}

int main(int argc, char **argv)
{
    std::mt19937 rng(argc > 1 ? atoi(argv[1]) : 1);
    const int count = argc > 2 ? atoi(argv[2]) : 1000;
    auto log = [&](double lo, double hi) { return (int)std::exp(std::uniform_real_distribution<double>(std::log(lo), std::log(hi + 0.5))(rng)); };
    for (int i = 0; i < count; ++i) {
        gconv_scan s{};
        s.groups = i % 2 ? 1 : log(1, 64);
        // the last channels that there are, or any number
        const int most = INT_MAX / s.groups, Cg = i % 4 < 2 ? most - log(1, 256) + 1 : log(1, most);
        s.C = s.groups * Cg;
        s.states = std::max(1, log(1, std::min(256.0, (double)INT_MAX / s.C)));
        s.L = log(1, std::max(1.0, std::min(500.0, std::ldexp(1.0, 40) / s.C)));
        s.N = log(1, std::max(1.0, std::min(3.0, std::ldexp(1.0, 40) / ((double)std::max(s.C, s.groups * s.states) * s.L))));
        if (!check_scan(&s, GCONV_BF16)) continue;
        look(s, false);
        look(s, true);
    }
    if (!last || plans < count) { printf("FAIL: %ld plans, %ld of the last channels\n", plans, last); ++errors; }
    printf("plans: %ld last: %ld errors: %ld\n", plans, last, errors);
    return errors ? 1 : 0;
}
