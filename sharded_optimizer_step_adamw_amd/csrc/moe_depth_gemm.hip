// moe_depth_gemm.hip -- the launches of the experts' weight gradients (the
// kernels: train_tiles.h).
#include "moe_internal.h"
#include "train_tiles.h"

namespace zopt {

hipError_t launch_depth(TgLaunch &L, hipStream_t stream) {
    return run_tile<kTgStore, true, true, kGroupDepth, false>(L, stream);
}

}  // namespace zopt
