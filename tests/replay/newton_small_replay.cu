// CPU replay of the cluster Newton-Schulz kernel's plan (newton_small.cu) over a range of sizes.  For every
// cluster the launch rule may take it walks a block's sweep as the kernel does, thread by thread, and checks
// that the values a thread keeps lie behind X and inside the block's shared memory, that X, A, S, R and the
// result's stage do too and in that order, and that where a kept value stands in R, the area the other blocks' shares land
// in, the plan orders the first share after the sweep that reads it.
// Usage: newton_small_replay <first m> <last m> <step of n>
#include "../../bwd_gconv_fwd_gb300/csrc/newton_small.cu"
#include <cstdio>
#include <cstdlib>
namespace gconv {
long long wait_limit() { return 1000000000LL; }
int num_sms() { return 152; }
}
using namespace gconv;
static long errors = 0, plans = 0, reach = 0;
#define CHECK(cond, ...) do { if (!(cond)) { if (errors++ < 10) { printf("FAIL: " __VA_ARGS__); printf("\n"); } } } while (0)

static void look(int rows, int cols)
{
    NewtonShape s{};
    s.G = 1; s.rows = rows; s.cols = cols;
    s.tall = rows > cols;
    s.m = s.tall ? cols : rows;
    s.n = s.tall ? rows : cols;
    for (int cs = 1; cs <= kMaxCluster; cs *= 2) {
        SmallParams p{};
        p.cluster = cs;
        p.slice = ((s.n + cs - 1) / cs + 63) / 64 * 64;
        if (p.slice > kMaxChunks * 64 || small_layout(s, cs, p.slice, &p) > kSmallSmem) continue;
        const int64_t room = (int64_t)small_plan(s, &p) - 1024;   // the kernel aligns its base to 1024 bytes
        ++plans;
        const int64_t sums = cs > 1 ? (int64_t)p.m16 * p.pitch : 0, a_bytes = (p.m16 + 63) / 64 * (int64_t)kChunkBytes;
        CHECK(p.oA == p.slice / 64 * kChunkBytes && p.oS == p.oA + a_bytes && p.oR >= p.oS + std::max(sums, a_bytes) &&
              p.oR + sums <= room, "%d x %d in %d: areas", rows, cols, cs);
        CHECK((int64_t)p.oOut + kSmallWarps * 32 * kSmallPitch * 4 <= room && (p.oOut != 0 || p.oA >= kSmallWarps * 32 * kSmallPitch * 4u),
              "%d x %d in %d: the result's stage", rows, cols, cs);
        CHECK(p.m16 % cs == 0, "%d x %d in %d: shares", rows, cols, cs);
        if (!p.keep) continue;
        // the block with the most columns, the first: its threads' kept items
        const int V = cols % 4 == 0 ? 4 : 1, width = std::min(p.slice, s.n);
        const int r_all = s.tall ? width : s.m, wide = s.tall ? s.m : width;
        int lpr = 1;
        while (lpr < 32 && lpr * V < wide) lpr <<= 1;
        const int rstep = kSmallThreads / lpr, cstep = lpr * V;
        int64_t end = p.oA;
        for (int tid : {0, lpr - 1, kSmallThreads - lpr, kSmallThreads - 1}) {
            int n = 0;
            for (int r = tid / lpr; r < r_all; r += rstep)
                for (int c = tid % lpr * V; ; c += cstep) {
                    if (c < wide) end = std::max<int64_t>(end, p.oA + ((int64_t)n * kSmallThreads + tid + 1) * V * 4);
                    ++n;
                    if (c + cstep >= wide) break;
                }
        }
        CHECK(end <= room, "%d x %d in %d: kept values end at %ld of %ld", rows, cols, cs, (long)end, (long)room);
        if (cs > 1 && end > p.oR) {
            ++reach;
            CHECK(p.ordered, "%d x %d in %d: kept values reach the shares (%ld > %u), which nothing orders", rows, cols, cs, (long)end,
                  p.oR);
        }
    }
}

int main(int argc, char **argv)
{
    if (argc != 4) {
        printf("usage: newton_small_replay <first m> <last m> <step of n>\n");
        return 2;
    }
    for (int m = atoi(argv[1]); m <= atoi(argv[2]); ++m)
        for (int n = m; n <= 8192; n += atoi(argv[3])) {
            look(m, n);
            if (n > m) look(n, m);
        }
    printf("plans: %ld, kept values in the shares' area: %ld\nerrors: %ld\n", plans, reach, errors);
    return errors != 0;
}
