// block_bwd_f32.cu -- the instances of block_bwd.cuh for f32 (a unit of its own for the build's sake).
#include "block_bwd.cuh"

namespace gconv {

void block_bwd_f32(int kind, const BlockShape &s, const BlockArgs &a, const StageMaps &maps, cudaStream_t st)
{
    launch_t<float>(kind, s, a, maps, st);
}

}  // namespace gconv
