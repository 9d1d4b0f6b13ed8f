// moe_gemm.hip -- the experts' products: the choice of tile and split, and the
// launches of the forward pass (the kernels: train_tiles.h).
#include "moe_internal.h"
#include "train_tiles.h"

namespace zopt {

int tile_height(int tile) { return tile == kTile64 ? 64 : tile == kTile128 ? 128 : 256; }
bool tile_seeks(int tile) { return seeks_rows(tile); }
void tile_shape(int tile, int32_t &height, int32_t &width, int32_t &rows, int32_t &cols) {
    auto set = [&](auto C) {
        height = C.BM;
        width = C.BN;
        rows = C.WR;
        cols = C.WC;
    };
    if (tile == kTile256) set(Cfg<kTile256>{});
    else if (tile == kTile256x128) set(Cfg<kTile256x128>{});
    else if (tile == kTile128) set(Cfg<kTile128>{});
    else set(Cfg<kTile64>{});
}

// As plan_tg, by figures of its own for a CU with all that it holds: with many
// rounds of tiles the caches bound the smaller ones, most where an operand is
// k-major, whose panels they read in more pieces.  The host does not know the
// groups' sizes: both kinds are chosen for groups of the average one, half a tile
// row of each unused (kGroupRows).
// kGroupDepth: a group of more than part_rows rows is summed in parts, which are
// joined afterwards.  One of twice the average, or of half of what a workgroup has
// to do in all, if that is more: else the largest group's tiles might run long
// after all others.  (With 13 experts of 4265 rows in all, of which one has 40%, the
// two gradients of 1000 x 602 matrices take 89 us without, 62 with parts.)
// Of eleven calls (16 to 2048 rows a group, reductions of 512 to 5632), each
// product forced to each kind of tile, the choice took at most 10% longer than
// the best but for some products under 30 us.
void plan_groups(TgEpilogue epi, TgGroups kind, bool b_km, TgLaunch &L) {
    constexpr int64_t cus = 256;
    static constexpr double stage[4][3] = {  // both row-major; B k-major; both
        {0.80, 0.81, 0.89}, {0.60, 0.50, 0.50}, {0.27, 0.35, 0.33}, {0.115, 0.20, 0.195}};
    const bool glu = epi == kTgGlu || epi == kTgMoeBack;
    const double rows = (double)L.M / L.groups;  // (kGroupRows)
    int all = L.prob[0].seg[0].stages;           // (kGroupDepth: of an average group)
    if (!glu && L.prob[0].nseg > 1) all += L.prob[0].seg[1].stages;
    double best = 0;
    L.splits = 1;
    for (int i = 0; i < 4; ++i) {
        const TileFigures &f = kTileFigures[i];
        const double busy = stage[i][kind == kGroupDepth ? 2 : b_km ? 1 : 0], each = glu ? f.heavy : f.plain;
        const int64_t bn = glu ? f.bn / 2 : f.bn, held = f.held * cus, across = (L.N + bn - 1) / bn;
        // `tiles` of `n` stages
        auto time = [&](int64_t tiles, int n) {
            const int64_t rounds = tiles / held, rest = tiles % held, left = (rest + cus - 1) / cus;
            auto load = [&](int64_t k) {
                const bool few = k == 1 && ((!glu && f.held > 1) || tiles < cus / 2);
                return few || f.alone > k * busy ? f.alone : k * busy;
            };
            return rounds * (n * load(f.held) + each) + (left ? n * load(left) + each : 0.0);
        };
        auto take = [&](double t, int64_t part) {
            if (best != 0 && t >= best) return;
            best = t;
            L.tile = f.tile;
            L.part_rows = (int32_t)part;
        };
        if (kind == kGroupRows) {
            const double high = rows <= f.bm / 2 ? 1.0 : rows / f.bm + 0.5;
            take(time((int64_t)((rows < 1 ? (double)L.M : high * L.groups) + 0.5) * across, all), 0);
            continue;
        }
        const int64_t per = (L.M + f.bm - 1) / f.bm * across * L.nprob;
        int64_t most = per * all * L.groups / held / 2 / 2 * 2;  // stages
        if (most < 2 * all) most = 2 * all;
        if (most < 8) most = 8;
        for (int split = 1; split <= 32; ++split) {
            int64_t part = split == 1 ? most : (all / 2 + split - 1) / split * 2;
            if (split > 1 && part >= most) continue;
            if (part < 8) break;
            const int64_t parts = all > part ? (all + part - 1) / part : 1;
            double t = time(per * L.groups * parts, (int)((all / 2 + parts - 1) / parts * 2));
            if (parts > 1) t += 4.0 + 8.0 * (double)(per * L.groups * parts * f.bm * f.bn) / 5.0e6;
            take(t, part > (1 << 24) ? (1 << 29) : part * 32);
        }
    }
}

// Scratch for the parts: a group of n > part_rows rows has less than 2 n /
// part_rows.
size_t group_part_bytes(const TgLaunch &L) {
    const int64_t bm = tile_height(L.tile), bn = L.tile == kTile256x128 ? 128 : bm;
    const int64_t per = (L.M + bm - 1) / bm * ((L.N + bn - 1) / bn) * L.nprob;
    return (size_t)(2 * (L.slots / L.part_rows) * per * bm * bn * 4);
}

hipError_t launch_rows_glu(bool gather, TgLaunch &L, hipStream_t stream) {
    return gather ? run_tile<kTgGlu, false, false, kGroupRows, true>(L, stream)
                  : run_tile<kTgGlu, false, false, kGroupRows, false>(L, stream);
}
hipError_t launch_rows(bool b_km, TgLaunch &L, hipStream_t stream) {
    return b_km ? run_tile<kTgRows, false, true, kGroupRows, false>(L, stream)
                : run_tile<kTgRows, false, false, kGroupRows, false>(L, stream);
}

}  // namespace zopt
