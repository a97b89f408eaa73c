// CPU replay of the causal convolution's work split (causal.cu, causal_shape and the walk of a worker) over random sizes: every
// element of every row falls to one lane of one worker, whatever place of 16 bytes the row begins at, the splits
// do not depend on the alignment, and no lane's first run begins more than a piece before its row.
// Usage: causal_walk_replay <seed> <count>
#include "../../bwd_gconv_fwd_gb300/csrc/causal.cu"
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
namespace gconv {
int num_sms() { return 152; }
}
static long errors = 0, shapes = 0;
#define CHECK(cond, what) do { if (!(cond)) { if (errors++ < 10) printf("FAIL: %s: N %d C %d L %d back %d whole %d\n", what, s.N, s.C, \
    s.L, back, whole); } } while (0)

static void look(const gconv_causal &s, gconv_dtype dt, bool back, bool whole)
{
    const CausalShape p = causal_shape(s, dt, back, whole);
    ++shapes;
    const int V = 16 / (dt == GCONV_BF16 ? 2 : 4), M = back ? kCausalBack : 2 * V, runs = back && p.segs > 1 ? p.TX - 1 : p.TX;
    CHECK(p.TX >= 1 && p.TX <= 32 && (p.TX & (p.TX - 1)) == 0 && p.segs >= 1 && p.splits >= 1 && runs >= 1, "lanes");
    CHECK(p.splits == causal_shape(s, dt, back, !whole).splits, "splits");
    CHECK(p.grid * (kCausalThreads / p.TX) >= (int64_t)s.C * p.splits, "workers");
    // one channel: how often its workers come by each piece
    const unsigned items = (unsigned)s.N * p.segs, all = (items + p.splits - 1) / p.splits;
    std::vector<int> seen(items, 0);
    for (int split = 0; split < p.splits; ++split) {
        const unsigned first = std::min<unsigned>(items, split * all), left = std::min(items - first, all);
        for (unsigned k = 0; k < left; ++k) ++seen[first + k];
    }
    for (unsigned i = 0; i < items; ++i) CHECK(seen[i] == 1, "pieces");
    for (int phase = 0; phase < (whole ? 1 : V); ++phase) {
        // runs of a row: from -phase on, M each, without a gap to the end
        const int64_t last = ((int64_t)(p.segs - 1) * runs + runs) * M - phase;
        CHECK(last >= s.L, "row");
    }
}

int main(int argc, char **argv)
{
    std::mt19937 rng(argc > 1 ? atoi(argv[1]) : 1);
    const int count = argc > 2 ? atoi(argv[2]) : 1000;
    auto log = [&](double lo, double hi) { return (int)std::exp(std::uniform_real_distribution<double>(std::log(lo), std::log(hi + 0.5))(rng)); };
    for (int i = 0; i < count; ++i) {
        gconv_causal s{};
        s.N = log(1, 256); s.C = log(1, 8192); s.L = log(1, 1 << 16); s.taps = 4;
        for (gconv_dtype dt : {GCONV_F32, GCONV_BF16})
            for (bool back : {false, true})
                for (bool whole : {false, true}) look(s, dt, back, whole);
    }
    printf("shapes: %ld errors: %ld\n", shapes, errors);
    return errors ? 1 : 0;
}
