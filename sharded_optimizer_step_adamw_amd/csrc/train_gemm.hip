// train_gemm.hip -- the products of the gradient operators over one problem:
// the choice of tile and split, and the launches (the kernels: train_tiles.h).
#include "train_tiles.h"

namespace zopt {

// Tile and split, by an estimate of the launch's time in microseconds from
// figures measured on the card (256 CUs):
//   stage   one workgroup alone on its CU takes `alone` a stage of 32, bound by
//           latency; a CU with all it holds (`held` of them) held * across, or
//           held * along with both operands row-major (256 x 128 tiles, whose
//           three buffers hold no pairs of stages, load halves of lines then)
//   tile    its first loads and its epilogue: `plain`, or `heavy` with
//           exponentials
//   split   a second launch (4) and 8 bytes an output and part at 5 TB/s
// Full rounds of tiles are computed whole; those left over, which would leave
// CUs idle, may be split along the reduction: [256, 50304] x [50304, 768]
// takes 937 us whole on 256 x 256 tiles, 54 us in 16 parts on 128 x 128, 39 us in
// the 21 parts that this chooses.
// Over 70 calls of drawn sizes each forced to one kind of tile, the choice took
// at most 5% longer than the best of the four but for six (6 to 13%, all but
// one of them under 100 us).
void plan_tg(TgEpilogue epi, TgLaunch &L) {
    constexpr int64_t cus = 256;  // (the figures' card; a launch takes the device's own count)
    const bool glu = epi == kTgGlu || epi == kTgGluBack;
    int all = L.prob[0].seg[0].stages;
    if (!glu && L.prob[0].nseg > 1) all += L.prob[0].seg[1].stages;
    double best = 0;
    for (const TileFigures &f : kTileFigures) {
        const int64_t bn = glu ? f.bn / 2 : f.bn, held = f.held * cus;
        const int64_t tiles = (L.M + f.bm - 1) / f.bm * ((L.N + bn - 1) / bn) * L.nprob;
        const int64_t rounds = tiles / held, rest = tiles % held;
        const bool plain = epi == kTgStore || epi == kTgSum;
        const double each = plain ? f.plain : f.heavy, busy = plain ? f.across : f.along;
        auto load = [&](int64_t n) {
            // (one on each of few CUs is not held up by the others; nor, across
            // lines, one where two would fit)
            const bool few = n == 1 && ((plain && f.held > 1) || tiles < cus / 2);
            return few || f.alone > n * busy ? f.alone : n * busy;
        };
        const double whole = rounds * (all * load(f.held) + each);
        for (int split = 1; split <= 32; ++split) {
            const int per = (all / 2 + split - 1) / split * 2;
            if (split > 1 && (per < 8 || rest == 0)) break;
            if ((all + per - 1) / per != split) continue;
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
    L.ldsum = (L.N + 3) / 4 * 4;
}

size_t tg_part_bytes(TgEpilogue epi, const TgLaunch &L) {
    if (L.splits == 1) return 0;
    const int64_t bm = L.tile == kTile64 ? 64 : L.tile == kTile128 ? 128 : 256;
    const int64_t bn = L.tile == kTile256x128 ? 128 : bm, bo = epi == kTgGlu || epi == kTgGluBack ? bn / 2 : bn;
    const int64_t tiles = (L.M + bm - 1) / bm * ((L.N + bo - 1) / bo) * L.nprob;
    return (size_t)((tiles - L.whole) * L.splits * bm * bn * 4);
}

hipError_t launch_tg(TgEpilogue epi, bool a_km, bool b_km, TgLaunch &L, hipStream_t stream) {
    if (epi == kTgXent) return run_tile<kTgXent, false, false>(L, stream);
    if (epi == kTgGlu) return run_tile<kTgGlu, false, false>(L, stream);
    if (epi == kTgGluBack) return run_tile<kTgGluBack, false, false>(L, stream);
    if (!b_km || (epi == kTgSum && !a_km)) return hipErrorInvalidValue;
    if (epi == kTgSum) return run_tile<kTgSum, true, true>(L, stream);
    return a_km ? run_tile<kTgStore, true, true>(L, stream) : run_tile<kTgStore, false, true>(L, stream);
}

}  // namespace zopt
