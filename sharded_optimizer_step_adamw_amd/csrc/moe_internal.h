// moe_internal.h -- declarations shared by routing and the experts' gated
// feed-forward (moe_route.hip, moe_rows.hip, moe_gemm.hip, moe_back_gemm.hip,
// moe_api.hip).
#pragma once

#include "train_internal.h"

namespace zopt {

constexpr int kMaxExperts = 1024, kMaxTop = 32;

// ---------------------------------------------------------------- routing

struct RouteArgs {
    int64_t tokens;
    int32_t experts, top, bf16, sigmoid, groups, top_groups, renormalise;
    float scale;
    const void *logits;   // fp32 or bf16 [tokens, experts], row stride ld
    int64_t ld;
    const float *bias;    // [experts] or NULL
    int32_t *chosen;      // [tokens, top]
    float *weights;       // [tokens, top]
    int32_t block_tokens;
    int32_t sort_here;    // (set by the launch) the one block, of all its threads, also sorts
    int32_t row_floats;   // (set by the launch) LDS of a token's ranges
    int32_t scored;       // ranks are scores and biases, not the logits
};
// Slots sorted by expert, stable: from the choice and the blocks' counts.
struct PlanArgs {
    int64_t tokens;
    int32_t experts, top, block_tokens;
    const int32_t *chosen;
    int32_t *counts, *total;  // [blocks, experts] and [experts] (blocks > 1)
    int32_t *offsets, *order, *place;
};
struct RouteBackArgs {
    int64_t tokens;
    int32_t experts, top, bf16, sigmoid, renormalise;
    float scale;
    const void *logits;
    int64_t ld;
    const int32_t *chosen;
    const float *dweights;
    void *dlogits;        // the logits' type, row stride lddl
    int64_t lddl;
};
// Tokens of a block (experts negative: that only sorts).
int32_t route_block_tokens(int64_t tokens, int32_t experts, int32_t groups, int32_t top, bool scored);
hipError_t launch_route(RouteArgs a, const PlanArgs &plan, hipStream_t stream);
hipError_t launch_plan_count(const PlanArgs &a, hipStream_t stream);
hipError_t launch_plan(const PlanArgs &a, hipStream_t stream);
hipError_t launch_route_back(const RouteBackArgs &a, hipStream_t stream);

// ---------------------------------------------------------------- experts

// What precedes the products, all in one launch:
//   kMoeTiles   the tile rows of height `height` (TgTileRow [1 + capacity]) from
//               the offsets
//   kMoeItems   the items of a sum over the experts' rows (TgItem [1 + experts + 2 (slots
//               / height)]) and the joins of their parts, of `height` rows at most (TgItem
//               [slots / height], no more than the experts): the parts, and behind
//               them the experts of one part, the largest first
//   kMoeShares  share [slots]: the slots' weights
//   kMoeGather  dst [slots, round8(cols)] = the slots' rows of src, zero beyond cols
//   kMoeCopy    dst [rows, round8(cols)] = src's rows, of which each
//               `group_rows` lie `group_stride` apart
enum MoePrepKind : int { kMoeTiles = 0, kMoeItems = 1, kMoeGather = 2, kMoeCopy = 3, kMoeShares = 4 };
struct MoePrep {
    int32_t kind;
    uint32_t blocks;              // set by the launch
    int32_t height, capacity;     // (capacity: of kMoeTiles)
    TgTileRow *tiles, *joins;
    int64_t rows, cols;
    const uint16_t *src;
    int64_t ld, group_rows, group_stride;
    uint16_t *dst;
    const float *weights;
    float *share;
};
constexpr int kMaxMoePreps = 12;
struct MoePrepList {
    MoePrep job[kMaxMoePreps];
    int32_t n;
    int32_t experts, top;
    int64_t slots;                // tokens * top
    const int32_t *offsets, *order;
};
hipError_t launch_moe_prep(MoePrepList &list, hipStream_t stream);

// out [tokens, cols] = the sums over a token's slots of weights (NULL: 1) times
// their rows [slots, cols] (of kTgRows: row stride ld, exponents' ldscale).  A slot without a place counts as zero.
// With dweights also what else ends a backward pass, in the same launch:
// dweights [tokens, top] = the sums of the slots' `parts` dots, and the joins of
// the weight gradients that were summed in parts.
struct MoeJoin {
    TgLaunch L;          // of which the part, items, joins, out, ldc, group_out, sizes
    int32_t rows, cols;  // waves of a tile across its rows and columns
    int32_t height, width;
    uint32_t blocks;     // (set by the launch)
};
struct MoeCombine {
    int64_t tokens, cols;
    int32_t top;
    int64_t slots;
    const int32_t *place;
    const float *weights;
    const uint16_t *rows;
    const uint8_t *scale;
    int64_t ld, ldscale;
    uint16_t *out;
    int64_t ldo;
    const float *dot;
    int64_t lddot;
    int32_t parts;
    float *dweights;
    MoeJoin join[2];
    uint32_t sum_blocks, dot_blocks;  // (set by the launch)
};
hipError_t launch_moe_combine(MoeCombine &c, hipStream_t stream);
hipError_t launch_fill_zero_groups(uint16_t *dst, int64_t ld, int64_t group_stride, int64_t groups, int64_t rows,
                                   int64_t cols, hipStream_t stream);

// The products (train_internal.h's kinds, over groups).
void plan_groups(TgEpilogue epi, TgGroups kind, bool b_km, TgLaunch &L);
int tile_height(int tile);
bool tile_seeks(int tile);  // finds the tile rows of 64 groups or less without a list
// rows and columns of a tile and its waves across them
void tile_shape(int tile, int32_t &height, int32_t &width, int32_t &rows, int32_t &cols);
size_t group_part_bytes(const TgLaunch &L);  // kGroupDepth
hipError_t launch_rows_glu(bool gather, TgLaunch &L, hipStream_t stream);      // kTgGlu
hipError_t launch_rows(bool b_km, TgLaunch &L, hipStream_t stream);            // kTgRows
hipError_t launch_rows_float(bool gather, TgLaunch &L, hipStream_t stream);    // kTgFloat, B k-major
hipError_t launch_rows_back(bool gather, TgLaunch &L, hipStream_t stream);     // kTgMoeBack
hipError_t launch_depth(TgLaunch &L, hipStream_t stream);                      // kTgStore, both k-major

}  // namespace zopt
