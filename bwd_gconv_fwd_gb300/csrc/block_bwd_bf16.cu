// block_bwd_bf16.cu -- the instances of block_bwd.cuh for bf16 (a unit of its own for the build's sake).
#include "block_bwd.cuh"

namespace gconv {

void block_bwd_bf16(int kind, const BlockShape &s, const BlockArgs &a, const StageMaps &maps, cudaStream_t st)
{
    launch_t<__nv_bfloat16>(kind, s, a, maps, st);
}

}  // namespace gconv
