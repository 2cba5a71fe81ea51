// Which of its three forms the greedy verify of drafted trees takes: host code, apart so that it can be tested.
#pragma once

#include <algorithm>

#include "sv_internal.h"

namespace sv {

// All rows, then the walk; depth by depth, the walk's rows alone; all in one launch, a tree to a workgroup.
enum TreeForm { TREE_ALL, TREE_LEVELS, TREE_SHORT };

constexpr int TREE_WAVES = 16;        // rows of a tree that a workgroup of the one launch reads side by side

// What decides between them, in us, from times of each: all rows are bound by the bytes or by
// workgroups of which each reads 16 KB or less; depth by depth adds a launch each; in one launch a compute unit
// reads its trees' rows by itself, a round of TREE_WAVES rows after another, a wave its row at a rate of its own,
// and all units together no faster than the card.  A call of two launches or more takes TREE_LEAST of the host,
// one of one launch TREE_LEAST_SHORT.
// Measured, drafts accepted 7 in 10, bfloat16 (trees, nodes, ids, depth: all rows, depth by depth, one launch):
//     1,  8,   1000, 4: 10.8, 20.0,  7.3      64, 16,   4000, 4: 11.1, 26.2,  7.7
//     1, 64,   4000, 8: 10.8, 29.8, 17.3     256, 64,   1000, 8: 53.1, 43.5, 12.3
//    16, 64, 128256, 8: 47.0, 41.0,  389     256, 16,   8000, 4: 21.1, 28.2, 13.5
//    32, 64,  32000, 8: 29.7, 42.6,  104     256, 64,   4000, 8: 53.1, 44.5, 22.9
//    64,  8, 128256, 4: 27.0, 33.1, 73.0     256, 64,   8000, 8: 56.3, 46.1, 41.4
//    64, 64, 128256, 8:  165, 49.2,  394     256, 16,  24000, 5: 37.6, 36.7, 31.9
//    64, 16,  16000, 5: 15.0, 35.5, 16.8     256, 16,  32000, 5: 48.1, 40.3, 42.5
//     1,  8,   1000, 0: 10.5,  9.8,  7.7      64,  1,  32000, 0: 10.6,  9.6, 16.7
//     1,  8, 128256, 0: 10.5,  9.4, 69.6       1,  1, 128256, 0: 10.5,  9.5, 48.6
constexpr double TREE_RATE = 6.5e6, TREE_UNIT_RATE = 4.5e4, TREE_WAVE_RATE = 4.2e3;   // bytes a us: the card, a
                                                                  // compute unit, a wave
constexpr double TREE_GROUP_US = 0.0026;                          // a workgroup among many
constexpr double TREE_ALL_US = 7.0, TREE_LEVEL_US = 4.0, TREE_SHORT_US = 4.0, TREE_ROUND_US = 1.0;
constexpr double TREE_LEAST = 10.5, TREE_LEAST_SHORT = 8.0;

inline TreeForm tree_form(int cus, int dtype, int B, int T, int V, int depth)
{
    const double row = (double)V * (dtype == 1 ? 2 : 4), us_bytes = (double)B * T * row / TREE_RATE;
    const int nch = num_chunks(NV_ARGMAX, dtype, V), rounds = (T + TREE_WAVES - 1) / TREE_WAVES;
    const double us_rows = std::max(us_bytes, (double)B * T * nch * TREE_GROUP_US);
    const double us_all = std::max(TREE_ALL_US + us_rows, TREE_LEAST);
    const double us_levels = std::max((depth + 2) * TREE_LEVEL_US + (depth + 1) * us_rows / T, TREE_LEAST);
    const double us_unit = rounds * TREE_ROUND_US + std::max((B + cus - 1) / cus * (T * row / TREE_UNIT_RATE),
                                                             rounds * row / TREE_WAVE_RATE);
    const double us_short = std::max(TREE_SHORT_US + std::max(us_unit, us_bytes), TREE_LEAST_SHORT);
    if (us_short < std::min(us_all, us_levels))
        return TREE_SHORT;
    return us_levels <= us_all ? TREE_LEVELS : TREE_ALL;
}

}  // namespace sv
