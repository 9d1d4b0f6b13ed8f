// The experts' products with the choice of tile and of parts in the hands of a
// test: the library's own source, whose plan_groups takes another name here, and
// a plan_groups that overrules it.  Built with the library's other sources of the
// experts into a library of its own.
#define plan_groups plan_groups_measured
#include "moe_gemm.hip"
#undef plan_groups

namespace zopt {

namespace {
int forced_tile = 0, forced_part = 0;
}

void plan_groups(TgEpilogue epi, TgGroups kind, bool b_km, TgLaunch &L);
void plan_groups(TgEpilogue epi, TgGroups kind, bool b_km, TgLaunch &L) {
    plan_groups_measured(epi, kind, b_km, L);
    if (forced_tile != 0) L.tile = forced_tile;
    if (kind == kGroupDepth && forced_part != 0) L.part_rows = forced_part;
}

}  // namespace zopt

// tile 0: the library's own choice; else 64, 128, 192 (256 x 128) or 256.  part 0: its
// own choice; else how many rows of an expert a part of its gradients sums at most,
// a multiple of 64.
extern "C" __attribute__((visibility("default"))) int force_moe_plan(int tile, int part) {
    using namespace zopt;
    if (tile != 0 && tile != kTile64 && tile != kTile128 && tile != kTile256x128 && tile != kTile256) return 1;
    if (part < 0 || part % 64 != 0) return 1;
    forced_tile = tile;
    forced_part = part;
    return 0;
}
