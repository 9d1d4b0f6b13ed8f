// moe_gemm.hip -- the experts' products: the choice of tile and split, and the
// launches of the forward pass (the kernels: train_tiles.h).
#include "moe_internal.h"
#include "train_tiles.h"

namespace zopt {
namespace {

template <int EPI, bool AKM, bool BKM, int GRP>
hipError_t run_tile(TgLaunch &L, hipStream_t stream) {
    if (L.tile == kTile256) return run<kTile256, EPI, AKM, BKM, GRP>(L, stream);
    if (L.tile == kTile256x128) return run<kTile256x128, EPI, AKM, BKM, GRP>(L, stream);
    if (L.tile == kTile128) return run<kTile128, EPI, AKM, BKM, GRP>(L, stream);
    return run<kTile64, EPI, AKM, BKM, GRP>(L, stream);
}

}  // namespace

int tile_height(int tile) { return tile == kTile64 ? 64 : tile == kTile128 ? 128 : 256; }

// As plan_tg.  The host does not know the groups' sizes, so both kinds are
// chosen for groups of the average one, half a tile row of each unused
// (kGroupRows), or of its reduction (kGroupDepth).
void plan_groups(TgEpilogue epi, TgGroups kind, TgLaunch &L) {
    constexpr int64_t cus = 256;
    const bool glu = epi == kTgGlu || epi == kTgMoeBack, plain = !glu;
    const double rows = (double)L.M / L.groups;  // (kGroupRows)
    int all = L.prob[0].seg[0].stages;
    if (!glu && L.prob[0].nseg > 1) all += L.prob[0].seg[1].stages;
    double best = 0;
    for (const TileFigures &f : kTileFigures) {
        const int64_t bn = glu ? f.bn / 2 : f.bn, held = f.held * cus, across = (L.N + bn - 1) / bn;
        int64_t tiles;
        if (kind == kGroupDepth) {
            tiles = (L.M + f.bm - 1) / f.bm * across * L.nprob * L.groups;
        } else {
            const double each = rows <= f.bm / 2 ? 1.0 : rows / f.bm + 0.5;
            tiles = (int64_t)((rows < 1 ? (double)L.M : each * L.groups) + 0.5) * across;
        }
        const int64_t rounds = tiles / held, rest = tiles % held;
        const double each = plain ? f.plain : f.heavy, busy = plain ? f.across : f.along;
        auto load = [&](int64_t n) {
            const bool few = n == 1 && ((plain && f.held > 1) || tiles < cus / 2);
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

hipError_t launch_rows_glu(TgLaunch &L, hipStream_t stream) {
    return run_tile<kTgGlu, false, false, kGroupRows>(L, stream);
}
hipError_t launch_rows_store(bool b_km, TgLaunch &L, hipStream_t stream) {
    return b_km ? run_tile<kTgStore, false, true, kGroupRows>(L, stream)
                : run_tile<kTgStore, false, false, kGroupRows>(L, stream);
}

}  // namespace zopt
