// moe_depth_gemm.hip -- the launches of the experts' weight gradients (the
// kernels: train_tiles.h).
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

hipError_t launch_depth(TgLaunch &L, hipStream_t stream) {
    return run_tile<kTgStore, true, true, kGroupDepth, false>(L, stream);
}

}  // namespace zopt
