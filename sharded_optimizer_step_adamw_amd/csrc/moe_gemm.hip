// moe_gemm.hip -- the experts' products: the choice of tile and split, and the
// launches of the forward pass (the kernels: train_tiles.h).
#include "moe_internal.h"
#include "train_tiles.h"

namespace zopt {
namespace {

template <int EPI, bool AKM, bool BKM, int GRP, bool LIST>
hipError_t run_tile(TgLaunch &L, hipStream_t stream) {
    if (L.tile == kTile256) return run<kTile256, EPI, AKM, BKM, GRP, LIST>(L, stream);
    if (L.tile == kTile256x128) return run<kTile256x128, EPI, AKM, BKM, GRP, LIST>(L, stream);
    if (L.tile == kTile128) return run<kTile128, EPI, AKM, BKM, GRP, LIST>(L, stream);
    return run<kTile64, EPI, AKM, BKM, GRP, LIST>(L, stream);
}

}  // namespace

int tile_height(int tile) { return tile == kTile64 ? 64 : tile == kTile128 ? 128 : 256; }

// As plan_tg, by figures of its own for a CU with all that it holds: with many
// rounds of tiles the caches bound the smaller ones, most where an operand is
// k-major, whose panels they read in more pieces.  The host does not know the
// groups' sizes: both kinds are chosen for groups of the average one, half a tile
// row of each unused (kGroupRows).
// Of eleven calls (16 to 2048 rows a group, reductions of 512 to 5632), each
// product forced to each kind of tile, the choice took at most 10% longer than
// the best but for some products under 30 us.
void plan_groups(TgEpilogue epi, TgGroups kind, bool b_km, TgLaunch &L) {
    constexpr int64_t cus = 256;
    static constexpr double stage[4][3] = {  // both row-major; B k-major; both
        {0.80, 0.81, 0.89}, {0.60, 0.50, 0.50}, {0.27, 0.35, 0.33}, {0.115, 0.20, 0.195}};
    const bool glu = epi == kTgGlu || epi == kTgMoeBack;
    const double rows = (double)L.M / L.groups;  // (kGroupRows)
    int all = L.prob[0].seg[0].stages;
    if (!glu && L.prob[0].nseg > 1) all += L.prob[0].seg[1].stages;
    double best = 0;
    for (int i = 0; i < 4; ++i) {
        const TileFigures &f = kTileFigures[i];
        const double busy = stage[i][kind == kGroupDepth ? 2 : b_km ? 1 : 0], each = glu ? f.heavy : f.plain;
        const int64_t bn = glu ? f.bn / 2 : f.bn, held = f.held * cus, across = (L.N + bn - 1) / bn;
        int64_t tiles;
        if (kind == kGroupDepth) {
            tiles = (L.M + f.bm - 1) / f.bm * across * L.nprob * L.groups;
        } else {
            const double high = rows <= f.bm / 2 ? 1.0 : rows / f.bm + 0.5;
            tiles = (int64_t)((rows < 1 ? (double)L.M : high * L.groups) + 0.5) * across;
        }
        const int64_t rounds = tiles / held, rest = tiles % held;
        auto load = [&](int64_t n) {
            const bool few = n == 1 && ((!glu && f.held > 1) || tiles < cus / 2);
            return few || f.alone > n * busy ? f.alone : n * busy;
        };
        const double whole = rounds * (all * load(f.held) + each);
        for (int split = 1; split <= (kind == kGroupDepth ? 32 : 1); ++split) {
            const int per = (all / 2 + split - 1) / split * 2;
            if (split > 1 && (per < 8 || rest == 0)) break;
            if (split > 1 && (all + per - 1) / per != split) continue;
            const int64_t on = (rest * split + cus - 1) / cus, full = on / f.held, left = on % f.held;
            double t = whole + full * (per * load(f.held) + each) + (left ? per * load(left) + each : 0.0);
            if (split > 1) t += 4.0 + 8.0 * split * (double)(rest * f.bm * f.bn) / 5.0e6;
            if (best == 0 || t < best) {
                best = t;
                L.tile = f.tile;
                L.splits = split;
                L.split_stages = per;
                L.whole = (int32_t)(split > 1 ? tiles - rest : tiles);
            }
        }
    }
}

size_t group_part_bytes(TgGroups kind, const TgLaunch &L) {
    if (kind == kGroupRows || L.splits == 1) return 0;
    const int64_t bm = tile_height(L.tile), bn = L.tile == kTile256x128 ? 128 : bm;
    const int64_t tiles = (L.M + bm - 1) / bm * ((L.N + bn - 1) / bn) * L.nprob * L.groups;
    return (size_t)((tiles - L.whole) * L.splits * bm * bn * 4);
}

hipError_t launch_rows_glu(bool gather, TgLaunch &L, hipStream_t stream) {
    return gather ? run_tile<kTgGlu, false, false, kGroupRows, true>(L, stream)
                  : run_tile<kTgGlu, false, false, kGroupRows, false>(L, stream);
}
hipError_t launch_rows_store(bool b_km, TgLaunch &L, hipStream_t stream) {
    return b_km ? run_tile<kTgStore, false, true, kGroupRows, false>(L, stream)
                : run_tile<kTgStore, false, false, kGroupRows, false>(L, stream);
}

}  // namespace zopt
