// moe_back_gemm.hip -- the launches of the experts' products over rows that only
// the backward pass makes (the kernels: train_tiles.h).
#include "moe_internal.h"
#include "train_tiles.h"

namespace zopt {

hipError_t launch_rows_float(bool gather, TgLaunch &L, hipStream_t stream) {
    return gather ? run_tile<kTgFloat, false, true, kGroupRows, true>(L, stream)
                  : run_tile<kTgFloat, false, true, kGroupRows, false>(L, stream);
}
hipError_t launch_rows_back(bool gather, TgLaunch &L, hipStream_t stream) {
    return gather ? run_tile<kTgMoeBack, false, false, kGroupRows, true>(L, stream)
                  : run_tile<kTgMoeBack, false, false, kGroupRows, false>(L, stream);
}

}  // namespace zopt
