// CPU replay of the causal convolution's numbering of workers (causal.cu, worker_of): the first and the last thread of a launch's
// blocks belong to the workers that 64-bit arithmetic gives, up to 2^31 channels.
// Usage: causal_worker_replay <seed> <count>
#include "../../bwd_gconv_fwd_gb300/csrc/causal.cu"
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>
namespace gconv {
int num_sms() { return 152; }
}

int main(int argc, char **argv)
{
    std::mt19937 rng(argc > 1 ? atoi(argv[1]) : 1);
    const int count = argc > 2 ? atoi(argv[2]) : 1000;
    long errors = 0, wide = 0;
    auto log = [&](double lo, double hi) { return (int)std::exp(std::uniform_real_distribution<double>(std::log(lo), std::log(hi + 0.5))(rng)); };
    for (int i = 0; i < count; ++i) {
        gconv_causal s{};
        s.N = 1; s.C = log(1, 2147483646.0); s.L = log(1, std::min(4096.0, std::ldexp(1.0, 40) / s.C)); s.taps = 4;
        for (gconv_dtype dt : {GCONV_F32, GCONV_BF16})
            for (bool back : {false, true}) {
                if (!check_causal(&s, dt)) { ++errors; continue; }
                const CausalShape p = causal_shape(s, dt, back, false);
                if (p.grid > INT_MAX) continue;
                wide += p.grid * kCausalThreads > UINT_MAX;
                for (int64_t block : {(int64_t)0, p.grid / 2, p.grid - 1})
                    for (int thread : {0, kCausalThreads - 1}) {
                        const int64_t want = (block * kCausalThreads + thread) / p.TX;
                        if (want > UINT_MAX || worker_of((unsigned)block, (unsigned)thread, (unsigned)p.TX) != want) ++errors;
                    }
            }
    }
    if (!wide) ++errors;
    printf("beyond 32 bits: %ld errors: %ld\n", wide, errors);
    return errors ? 1 : 0;
}
