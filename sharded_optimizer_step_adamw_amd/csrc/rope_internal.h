// rope_internal.h -- declarations of the norms and rotation of queries and
// keys (rope.hip, rope_api.hip).
#pragma once

#include "train_internal.h"

namespace zopt {

// One of the two inputs, [tokens, heads, width] with strides of its own.
struct RopeSide {
    const uint16_t *x, *dy;
    uint16_t *out;        // y, or dx
    int64_t xt, xh, dt, dh, ot, oh;  // strides between tokens and between heads
    const uint16_t *w;    // [width] or NULL
    uint16_t *dw;         // [width]
    int32_t heads;
};
struct RopeArgs {
    RopeSide side[2];     // queries, keys (heads 0: none)
    int64_t tokens, positions;
    int32_t width, rot, pairs;
    float eps;
    const float2 *table;  // [positions, rot / 2]: cosine, sine
    const int64_t *position;  // [tokens], or NULL: the token's number
    float *part;          // [blocks, width]: sums of dw, the queries' blocks first
    int32_t group;        // lanes of a row (set by the launch)
    int32_t first_blocks; // blocks of the queries
    int32_t blocks;
};
// Sets group and the blocks.
void plan_rope(RopeArgs &a);
hipError_t launch_rope(const RopeArgs &a, hipStream_t stream);
hipError_t launch_rope_back(const RopeArgs &a, hipStream_t stream);
hipError_t launch_rope_table(int64_t positions, int32_t rot, double base, float2 *table, hipStream_t stream);

constexpr int kMaxHeadWidth = 512;

}  // namespace zopt
