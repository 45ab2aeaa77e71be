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

}  // namespace moe
