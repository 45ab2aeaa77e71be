// How the TMA boxes of a bf16 operand move along K (ffn_map, ffn_map_mn).
#pragma once

#include "ffn_block.h"

namespace moe {

// Coordinates of an operand's box of 128 rows of M (or N) from m0 on: the
// first K block's, and the step per K block; two: the tile takes two boxes.
struct BoxWalk {
    int c0, c1, c2, d0, d1;
    bool two;
    __device__ __forceinline__ BoxWalk(int order, int m0)
        : c0(order == MN_ROWS ? m0 / 2 : 0),
          c1(order == K_MAJOR ? m0 : 0),
          c2(order == MN_BLOCKS ? m0 / 64 : 0),
          d0(order == K_MAJOR ? 32 : 0),
          d1(order == K_MAJOR ? 0 : 64),
          two(order == MN_ROWS) {}
};

// Where the saved act(g) and u act'(g) of row r, column c lie (floats), for rows
// of n columns: blocks of 32 x 32 one after another, a block's columns in
// groups of 8, 32 bytes of each row after another.  A warp whose lanes hold a
// row each then reads and writes whole lines.  (Row-major, the saves of 4096 x
// 8192 took 60 us beside their products' 145, and reading them 40 beside 87.)
__host__ __device__ inline size_t saved_at(size_t r, size_t c, size_t n) {
    return ((r >> 5) * ((n + 31) >> 5) + (c >> 5)) * 1024 + ((c >> 3) & 3) * 256 + (r & 31) * 8 + (c & 7);
}
inline size_t saved_floats(size_t m, size_t n) { return ((m + 31) / 32) * ((n + 31) / 32) * 1024; }

}  // namespace moe
