// moe_back_gemm.hip -- the launches of the experts' products that only the
// backward pass makes (the kernels: train_tiles.h).
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

hipError_t launch_rows_float(TgLaunch &L, hipStream_t stream) {
    return run_tile<kTgFloat, false, true, kGroupRows>(L, stream);
}
hipError_t launch_rows_back(TgLaunch &L, hipStream_t stream) {
    return run_tile<kTgMoeBack, false, false, kGroupRows>(L, stream);
}
hipError_t launch_depth(TgLaunch &L, hipStream_t stream) {
    return run_tile<kTgStore, true, true, kGroupDepth>(L, stream);
}

}  // namespace zopt
