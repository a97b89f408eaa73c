// block_internal.h -- what the block norm / block join translation units share.
#pragma once

#include "block_norm.cuh"

namespace gconv {

// The shape of one launch (block_norm.cu, block_shape).
struct BlockShape {
    int row, held;            // the kernels of block_row.cuh; channels a thread holds
    int staged;               // the kernels of block_stage.cuh, with:
    int PT, flat, per, total, stages, cluster, Cc, pitch, tensor, boxes, box_rows, pieces;
    int vec;                  // positions a thread holds at once
    int TX, TY, Z, tiles, splits;
    int images;               // of the channel sums a backward call keeps: N, or 1
    int threads;
    unsigned grid;
    size_t smem;
};

enum { kBlockNorm = 0, kBlockJoin = 1, kBlockJoinNext = 2 };

constexpr size_t kBlockSmem = 227 * 1024 - 128;   // beside the kernels' barriers

void block_fwd_bf16(int kind, const BlockShape &s, const BlockArgs &a, const StageMaps &maps, cudaStream_t st);
void block_fwd_f32(int kind, const BlockShape &s, const BlockArgs &a, const StageMaps &maps, cudaStream_t st);
void block_bwd_bf16(int kind, const BlockShape &s, const BlockArgs &a, const StageMaps &maps, cudaStream_t st);
void block_bwd_f32(int kind, const BlockShape &s, const BlockArgs &a, const StageMaps &maps, cudaStream_t st);

}  // namespace gconv
