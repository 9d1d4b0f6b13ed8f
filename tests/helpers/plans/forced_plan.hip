// The products of the gradient operators with the choice of tile and split in
// the hands of a test: the library's own source, whose plan_tg takes another
// name here, and a plan_tg that overrules it.  Built with the library's
// train_api.hip and train_rows.hip into a library of its own.
#define plan_tg plan_tg_measured
#include "train_gemm.hip"
#undef plan_tg

namespace zopt {

namespace {
int forced_tile = 0, forced_splits = 1, forced_rest = 0;
}

void plan_tg(TgEpilogue epi, TgLaunch &L) {
    plan_tg_measured(epi, L);
    if (forced_tile == 0) return;
    const bool glu = epi == kTgGlu || epi == kTgGluBack;
    int all = L.prob[0].seg[0].stages;
    if (!glu && L.prob[0].nseg > 1) all += L.prob[0].seg[1].stages;
    const int64_t bm = forced_tile == kTile64 ? 64 : forced_tile == kTile128 ? 128 : 256;
    const int64_t bn = forced_tile == kTile256x128 ? 128 : bm, bo = glu ? bn / 2 : bn;
    const int64_t tiles = (L.M + bm - 1) / bm * ((L.N + bo - 1) / bo) * L.nprob;
    L.tile = forced_tile;
    // parts are whole pairs of stages
    L.split_stages = (all / 2 + forced_splits - 1) / forced_splits * 2;
    L.splits = (all + L.split_stages - 1) / L.split_stages;
    // the last forced_rest / 2 of the tiles are split
    L.whole = (int32_t)(L.splits > 1 ? tiles - (tiles * forced_rest + 1) / 2 : tiles);
    if (L.whole == tiles) {
        L.splits = 1;
        L.split_stages = all;
    }
}

}  // namespace zopt

// tile 0: the library's own choice; else 64, 128, 192 (256 x 128) or 256, the
// reduction of all tiles (rest 2), half of them (1) or none (0) in `splits` parts.
extern "C" __attribute__((visibility("default"))) int force_plan(int tile, int splits, int rest) {
    using namespace zopt;
    if (tile != 0 && tile != kTile64 && tile != kTile128 && tile != kTile256x128 && tile != kTile256) return 1;
    if (splits < 1 || splits > 32 || rest < 0 || rest > 2) return 1;
    forced_tile = tile;
    forced_splits = splits;
    forced_rest = rest;
    return 0;
}
