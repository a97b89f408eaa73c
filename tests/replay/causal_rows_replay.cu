// CPU replay of a causal convolution worker's way through its rows (causal.cu: causal_shape, Walk and its steps as the kernels make
// them) over random sizes, lengths and places of the rows within 16 bytes: every element of every sequence falls to
// one lane in one round, the row's pointers go along with the sequence's number and its length, the first run of a row begins
// less than a 16-byte piece before it, and all workers of a warp make the same number of rounds.
// Usage: causal_rows_replay <seed> <count>
#include "../../bwd_gconv_fwd_gb300/csrc/causal.cu"
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
namespace gconv {
int num_sms() { return 152; }
}
static long errors = 0, shapes = 0, longer = 0, crossing = 0, narrow = 0;
#define CHECK(cond, what) do { if (!(cond)) { if (errors++ < 10) printf("FAIL: %s: N %d C %d L %d back %d whole %d\n", what, s.N, s.C, \
    s.L, back, whole); } } while (0)

static void look(const gconv_causal &s, gconv_dtype dt, bool back, bool whole, std::mt19937 &rng)
{
    const CausalShape p = causal_shape(s, dt, back, whole);
    ++shapes;
    const int V = 16 / (dt == GCONV_BF16 ? 2 : 4), M = back ? kCausalBack : 2 * V, runs = back && p.segs > 1 ? p.TX - 1 : p.TX;
    std::vector<int> lengths(s.N), phases(s.N);
    for (int n = 0; n < s.N; ++n) {
        lengths[n] = (int)(rng() % (s.L + 3)) - 1;
        phases[n] = whole ? 0 : rng() % V;
    }
    CausalArgs a{};
    causal_args(s, &a);
    a.TX = p.TX; a.segs = p.segs; a.splits = p.splits; a.lengths = lengths.data();
    std::vector<std::vector<unsigned char>> seen(s.N, std::vector<unsigned char>(s.L, 0));
    unsigned rounds = 0;
    for (int split = 0; split < p.splits; ++split) {
        Walk at(a, split, s.C - 1, true);
        at.t = (int64_t)at.seg * runs * M;
        if (split == 0) rounds = at.all;
        CHECK(at.all == rounds, "rounds");
        longer += at.left > 1;
        int row = at.n, made = 0, begun = at.n;         // the sequence that the kernels' pointers are at
        for (; at.made < at.all; at.step(a, runs * M, [&] { ++row; }), ++made) {
            if (!at.on) {
                CHECK(at.end == 0, "end of no sequence");
                continue;
            }
            crossing += at.n != begun;
            begun = at.n;
            CHECK(at.n >= 0 && at.n < s.N && row == at.n, "row");
            if (at.n < 0 || at.n >= s.N) break;
            CHECK(at.end == std::min(std::max(lengths[at.n], 0), s.L), "length");
            CHECK(at.t == (int64_t)at.seg * runs * M && at.seg < p.segs, "piece");
            for (int tx = 0; tx < runs; ++tx) {
                const int64_t t = at.t + (int64_t)tx * M - phases[at.n];
                CHECK(t > -V, "first run");
                for (int64_t j = std::max<int64_t>(t, 0); j < std::min<int64_t>(t + M, s.L); ++j) ++seen[at.n][j];
            }
        }
        CHECK(made == (int)rounds, "rounds made");
    }
    narrow += p.TX < 32 && rounds > 1;
    for (int n = 0; n < s.N; ++n)
        for (int t = 0; t < s.L; ++t) CHECK(seen[n][t] == 1, "element");
}

int main(int argc, char **argv)
{
    std::mt19937 rng(argc > 1 ? atoi(argv[1]) : 1);
    const int count = argc > 2 ? atoi(argv[2]) : 1000;
    auto log = [&](double lo, double hi) { return (int)std::exp(std::uniform_real_distribution<double>(std::log(lo), std::log(hi + 0.5))(rng)); };
    for (int i = 0; i < count; ++i) {
        gconv_causal s{};
        s.N = log(1, 64); s.C = log(1, 32768); s.L = log(1, 5000); s.taps = 4;
        for (gconv_dtype dt : {GCONV_F32, GCONV_BF16})
            for (bool back : {false, true})
                for (bool whole : {false, true}) look(s, dt, back, whole, rng);
    }
    // the sizes reach workers of several pieces, of several rows, and of less than a warp
    if (!longer || !crossing || !narrow) ++errors;
    printf("shapes: %ld several pieces: %ld several rows: %ld part of a warp: %ld errors: %ld\n", shapes, longer, crossing, narrow, errors);
    return errors ? 1 : 0;
}
