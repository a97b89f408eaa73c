// block_internal.h -- what the block norm / block join translation units share.
#pragma once

#include "block_norm.cuh"

namespace gconv {

// The shape of one launch (block_norm.cu, block_shape).
struct BlockShape {
    int vec, one;             // positions a thread holds at once; a thread's channels fit in registers
    int TX, TY, Z, PV, tiles, splits;
    int threads;
    unsigned grid;
    size_t smem;
};

enum { kBlockNorm = 0, kBlockJoin = 1, kBlockJoinNext = 2 };

// Channels a thread holds: four where it holds 4 or 8 positions of each, eight where 1 or 2.
constexpr int block_nch(int vec) { return vec >= 4 ? 4 : 8; }

void block_fwd_launch(int kind, gconv_dtype dt, const BlockShape &s, const BlockArgs &a, cudaStream_t st);
void block_bwd_launch(int kind, gconv_dtype dt, const BlockShape &s, const BlockArgs &a, cudaStream_t st);

}  // namespace gconv
