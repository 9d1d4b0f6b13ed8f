// tile_walk.h -- the order in which the products walk their tiles.
#pragma once

#include "train_internal.h"

namespace zopt {
namespace {

// Tile t of a tiles_m x tiles_n grid: bands of 16 tile rows, in a band groups
// of 8 columns, in a group runs of 4 rows, column by column.  A round of 256
// tiles is then about 16 x 16 and an XCD's 32 about 4 x 8: few operand panels
// in each L2, and few of them read more than once from HBM.
__device__ __forceinline__ void tile_at(int t, int tm, int tn, int &ti, int &tj) {
    const int band = t / (16 * tn), r0 = band * 16;
    t -= band * 16 * tn;
    const int h = tm - r0 < 16 ? tm - r0 : 16;
    const int group = t / (8 * h), c0 = group * 8;
    t -= group * 8 * h;
    const int w = tn - c0 < 8 ? tn - c0 : 8;
    const int run = t / (4 * w), q0 = run * 4;
    t -= run * 4 * w;
    const int hh = h - q0 < 4 ? h - q0 : 4;
    tj = c0 + t / hh;
    ti = r0 + q0 + t % hh;
}

// Tile t of an item's, kGroupDepth: the problems side by side
__device__ __forceinline__ void item_tile(const TgLaunch &L, int t, int &prob, int &ti, int &tj) {
    const int per = L.tiles_m * L.tiles_n;
    prob = t >= per ? 1 : 0;
    tile_at(t - prob * per, L.tiles_m, L.tiles_n, ti, tj);
}

}  // namespace
}  // namespace zopt
