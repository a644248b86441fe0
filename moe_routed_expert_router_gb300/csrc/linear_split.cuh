// How a product of linear.cu is shared by blocks, warps and passes over a block's rows.  Plain C++: tests compile it
// without CUDA and run it over the sizes.
#pragma once

#include <limits.h>

#include <algorithm>

#include "card.cuh"

#ifdef __CUDACC__
#define MOE_BOTH __host__ __device__
#else
#define MOE_BOTH
#endif

namespace moe {

// Of a product whose blocks take 8 * nt tokens (nt 1, 2 or 4).
constexpr int linear_tokens(int T) { return T <= 8 ? 1 : T <= 16 ? 2 : 4; }
// Values of K a stage: 256, and half of it where 32 tokens have to share the registers.
constexpr int linear_stage_k(int nt) { return nt >= 4 ? 128 : 256; }
// Warps of a block: what the tokens' registers leave room for.
constexpr int linear_warps(int nt) { return nt == 1 ? 16 : 12; }
constexpr int kLinearRows = 16;            // rows a tile (32 took the sums' place from the ring: 53 us against 47 at 1 x 100003 x 4096, before linear_tc.cu had that size)
constexpr int kScaleBytes = 16;            // a row's place for a stage's scales (MXFP4 uses half)
constexpr int kCodePad = 16;               // behind a row's codes: eight rows' equal words lie in different banks
constexpr int kLeastLinearRing = 2, kMostLinearRing = 6;
// Bytes of a warp's stage of a tile, and of its sums of one.
constexpr int linear_stage_bytes(int nt) { return kLinearRows * (linear_stage_k(nt) / 2 + kCodePad + kScaleBytes); }
constexpr int linear_sum_bytes(int nt) { return nt * 512; }

struct LinearSplit {
    int blocks, groups;                    // blocks that share the rows, and groups of tokens: the grid
    int base, extra;                       // rows of a block: base, and one more in the first `extra` blocks
    int passes, pass_rows, tile_rows;      // over a block's rows; rows a pass and a tile
    int wk, wm, tiles;                     // warps that share K; groups of them, which share a pass's tiles; tiles a group
    int ring;                              // stages of a warp's ring
    int smem;                              // bytes a block
};

inline LinearSplit linear_split(int nt, int T, int N, int K) {
    const size_t stage = linear_stage_bytes(nt), join = linear_sum_bytes(nt);
    const int most_warps = linear_warps(nt), stages = blocks_of(K, linear_stage_k(nt));
    LinearSplit s{};
    s.groups = blocks_of(T, 8 * nt);
    s.blocks = std::min(std::max(1, kSms / s.groups), N);
    const int rows = blocks_of(N, s.blocks);
    s.base = N / s.blocks;
    s.extra = N % s.blocks;
    // the split with the shortest longest share: stages, each taking its tokens (about three tiles of work) and its tiles
    const int all = blocks_of(rows, kLinearRows);
    int best = INT_MAX;
    for (int wk = std::min(stages, most_warps); wk >= 1; --wk) {
        const int wm = std::min(most_warps / wk, all), cost = blocks_of(stages, wk) * (3 + blocks_of(all, wm));
        if (cost < best) {
            best = cost;
            s.wk = wk;
            s.wm = wm;
        }
    }
    const int warps = s.wk * s.wm;
    const int most = (int)((kSmemBlock / warps - kLeastLinearRing * stage) / join);    // tiles of a warp in a pass
    s.passes = blocks_of(rows, s.wm * most * kLinearRows);
    s.pass_rows = blocks_of(rows, s.passes);
    s.passes = blocks_of(rows, s.pass_rows);       // rounding up may have emptied the last ones
    s.tiles = blocks_of(s.pass_rows, s.wm * kLinearRows);
    s.tile_rows = blocks_of(s.pass_rows, s.wm * s.tiles);
    s.ring = (int)std::min<size_t>(kMostLinearRing, (kSmemBlock / warps - s.tiles * join) / stage);
    s.smem = (int)(warps * (s.ring * stage + s.tiles * join));
    return s;
}

// Rows `first` up to `end`.
struct RowRange {
    int first, end;
};

// Rows of a block.
MOE_BOTH inline RowRange linear_block_rows(const LinearSplit &s, int block) {
    const int first = block * s.base + std::min(block, s.extra);
    return {first, first + s.base + (block < s.extra)};
}

// Rows of a block's pass, and of tile `tile` (of wm * tiles) of those.  Only lengths are compared and added up to where
// rows are: a pass that there is starts at most at the block's end, so nothing passes 32 bits for the largest N.
MOE_BOTH inline RowRange linear_pass_rows(const LinearSplit &s, RowRange block, int pass) {
    const int first = block.first + std::min(pass * s.pass_rows, block.end - block.first);
    return {first, first + std::min(s.pass_rows, block.end - first)};
}
MOE_BOTH inline RowRange linear_tile_rows(const LinearSplit &s, RowRange pass, int tile) {
    const int first = pass.first + std::min(tile * s.tile_rows, pass.end - pass.first);
    return {first, first + std::min(s.tile_rows, pass.end - first)};
}

}  // namespace moe
