// moe_api.hip -- the C-ABI entry points of routing and the experts' gated
// feed-forward (declared in zopt.h).
#include <cmath>

#include "moe_internal.h"
#include "train_api.h"

namespace zopt {
namespace {

constexpr int64_t kMaxSlots = (int64_t)1 << 30;  // tokens * top: their numbers are 32 bits wide
constexpr int32_t kMaxRanges = 64;

zopt_status check_route(int64_t T, int32_t E, int32_t k) {
    if (!range(T, 0, kMaxRows) || !range(E, 1, kMaxExperts) || !range(k, 1, kMaxTop < E ? kMaxTop : E))
        return ZOPT_ERR_SIZE;
    return T * k <= kMaxSlots ? ZOPT_OK : ZOPT_ERR_SIZE;
}
// The sort's workspace for blocks of `each` tokens: their counts and the
// experts' totals.
size_t plan_bytes(int64_t T, int32_t E, int32_t each) {
    const int64_t blocks = (T + each - 1) / each;
    return blocks > 1 ? (size_t)up((blocks + 1) * E * 4, 256) : 0;
}
PlanArgs plan_args(int64_t T, int32_t E, int32_t k, int32_t each, const int32_t *chosen, void *workspace,
                   int32_t *offsets, int32_t *order, int32_t *place) {
    int32_t *counts = static_cast<int32_t *>(workspace);
    return PlanArgs{T, E, k, each, chosen, counts, counts + (T + each - 1) / each * E, offsets, order, place};
}

// A weight [experts, rows, cols] as the products read it, in place or a padded
// copy.
struct Weight {
    const uint16_t *p;
    int64_t ld, group;  // strides of rows and experts
    bool copy;
    size_t at;
};
bool weight_needs_copy(const uint16_t *p, int64_t ld, int64_t group, int64_t cols) {
    return !aligned16(p) || (ld & 7) || (group & 7) || (cols & 7) || ld > kMaxStride;
}
Weight weight(const uint16_t *p, int64_t ld, int64_t group, int64_t experts, int64_t rows, int64_t cols, bool force,
              Carve &c) {
    Weight w{p, ld, group, false, 0};
    w.copy = force || weight_needs_copy(p, ld, group, cols);
    if (w.copy) {
        w.ld = up(cols, 8);
        w.group = rows * w.ld;
        w.at = c.take(experts * w.group * 2);
    }
    return w;
}

// A matrix [tokens, cols] whose rows the products take by expert: gathered as it
// lies, or from a copy in the slots' order (row stride up(cols, 8)): where it
// is not aligned, where it spans more than the products' 32-bit offsets reach,
// and for the weight gradients.
struct Rows {
    const uint16_t *p, *slots;
    int64_t ld;
    bool gathered, copy;
    size_t at;
};
Rows token_rows(const uint16_t *p, int64_t ld, int64_t tokens, int64_t top, int64_t cols, bool copy, Carve &c) {
    Rows r{p, nullptr, ld, false, copy, 0};
    r.gathered = aligned16(p) && !(ld & 7) && !(cols & 7) && ld <= kMaxStride &&
                 ((tokens - 1) * ld + cols) * 2 <= kGatherBytes;
    r.copy = copy || !r.gathered;
    if (r.copy) r.at = c.take(tokens * top * up(cols, 8) * 2);
    return r;
}

// What a call does, from its sizes alone: both the size query and the call make
// it.
struct MoePlan {
    int64_t S, T, D, F, Dp, Fp;
    int32_t E, k;
    bool back;
    Weight wg, wu, wd;
    Rows x, dy;
    size_t share, h, dh, dg, du, rows, scale, dot, total;
    int64_t scales;  // exponents of a slot's row
    int64_t parts;  // dots of a slot
    size_t tiles[3], items[2], joins[2], part[2];
    TgLaunch glu, down, dhf, dx, dwgu, dwd;

    TgLaunch launch(int64_t M, int64_t N) const {
        TgLaunch L{};
        L.nprob = 1;
        L.prob[0].nseg = 1;
        L.M = (int32_t)M;
        L.N = (int32_t)N;
        L.groups = E;
        L.slots = (int32_t)S;
        L.tokens = (int32_t)T;
        return L;
    }
    static TgSegment segment(TgOperand a, TgOperand b) {
        const int32_t n = a.k > b.k ? a.k : b.k;
        return TgSegment{a, b, (n + 63) / 64 * 2};
    }
    // operands: the slots' rows along the reduction and across it, a weight's
    TgOperand slots_along(const void *p, int64_t ld, int64_t cols) const {
        return TgOperand{static_cast<const uint16_t *>(p), ld, (int32_t)S, (int32_t)up(cols, 8)};
    }
    TgOperand rows_along(const Rows &r, int64_t cols) const {
        return r.gathered ? slots_along(r.p, r.ld, cols) : slots_along(r.slots, up(cols, 8), cols);
    }
    TgOperand slots_across(const void *p, int64_t ld, int64_t cols) const {
        return TgOperand{static_cast<const uint16_t *>(p), ld, (int32_t)up(cols, 8), (int32_t)S};
    }
    static TgOperand along(const Weight &w, int64_t rows, int64_t cols) {
        return TgOperand{w.p, w.ld, (int32_t)rows, (int32_t)up(cols, 8)};
    }
    static TgOperand across(const Weight &w, int64_t rows, int64_t cols) {
        return TgOperand{w.p, w.ld, (int32_t)up(cols, 8), (int32_t)rows};
    }
    // tile rows of a launch's height
    int64_t capacity(const TgLaunch &L) const { return S / tile_height(L.tile) + (E < S ? E : S); }
    // the reduction of an average expert, for the choice of tile and split
    int32_t average() const { return (int32_t)((S / E + 63) / 64 * 2); }
};

MoePlan moe_plan(int64_t T, int64_t D, int64_t F, int32_t E, int32_t k, const uint16_t *x, int64_t ldx,
                 const uint16_t *dy, int64_t lddy, const uint16_t *wg, const uint16_t *wu,
                 int64_t ldw, int64_t groupw, const uint16_t *wd, int64_t ldd, int64_t groupd, bool back) {
    MoePlan p{};
    Carve c;
    p.T = T;
    p.D = D;
    p.F = F;
    p.E = E;
    p.k = k;
    p.S = T * k;
    p.Dp = up(D, 8);
    p.Fp = up(F, 8);
    p.back = back;
    const int64_t S = p.S;
    // (the products take both with one layout)
    const bool copy = weight_needs_copy(wg, ldw, groupw, D) || weight_needs_copy(wu, ldw, groupw, D);
    p.wg = weight(wg, ldw, groupw, E, F, D, copy, c);
    p.wu = weight(wu, ldw, groupw, E, F, D, copy, c);
    p.wd = weight(wd, ldd, groupd, E, D, F, false, c);
    if (S == 0) {
        p.total = c.total();
        return p;
    }
    p.x = token_rows(x, ldx, T, k, D, back, c);
    p.h = c.take(S * p.Fp * 2);
    p.rows = c.take(S * p.Dp * 2);
    p.scales = (D + kRowsGroup - 1) / kRowsGroup;
    p.scale = c.take(S * p.scales);
    p.glu = p.launch(S, F);
    p.glu.prob[0].seg[0].stages = (int32_t)((p.Dp + 63) / 64 * 2);
    plan_groups(back ? kTgMoeBack : kTgGlu, kGroupRows, false, p.glu);
    if (!back) {
        p.down = p.launch(S, D);
        p.down.prob[0].seg[0].stages = (int32_t)((p.Fp + 63) / 64 * 2);
        plan_groups(kTgRows, kGroupRows, false, p.down);
    } else {
        p.dy = token_rows(dy, lddy, T, k, D, true, c);
        p.share = c.take(S * 4);
        p.dh = c.take(S * p.Fp * 4);
        p.dg = c.take(S * p.Fp * 2);
        p.du = c.take(S * p.Fp * 2);
        p.parts = (F + 31) / 32;
        p.dot = c.take(S * p.parts * 4);
        p.dhf = p.launch(S, F);
        p.dhf.prob[0].seg[0].stages = (int32_t)((p.Dp + 63) / 64 * 2);
        plan_groups(kTgFloat, kGroupRows, true, p.dhf);
        p.dx = p.launch(S, D);
        p.dx.prob[0].nseg = 2;
        p.dx.prob[0].seg[0].stages = p.dx.prob[0].seg[1].stages = (int32_t)((p.Fp + 63) / 64 * 2);
        plan_groups(kTgRows, kGroupRows, true, p.dx);
        p.dwgu = p.launch(F, D);
        p.dwgu.nprob = 2;
        p.dwgu.prob[0].seg[0].stages = p.average();
        plan_groups(kTgStore, kGroupDepth, true, p.dwgu);
        p.dwd = p.launch(D, F);
        p.dwd.prob[0].seg[0].stages = p.average();
        plan_groups(kTgStore, kGroupDepth, true, p.dwd);
        int i = 0;
        for (TgLaunch *L : {&p.dwgu, &p.dwd}) {
            // (groups of more than part_rows rows, and the parts of all of them)
            const int64_t splits = S / L->part_rows;
            L->join_limit = (int32_t)(splits < E ? splits : E);
            L->item_limit = (int32_t)(E + 2 * splits);
            p.part[i] = c.take(group_part_bytes(*L));
            p.items[i] = c.take((1 + L->item_limit) * (int64_t)sizeof(TgItem));
            p.joins[i++] = c.take((L->join_limit + 1) * (int64_t)sizeof(TgItem));
        }
    }
    const TgLaunch *rows[3] = {&p.glu, back ? &p.dhf : &p.down, back ? &p.dx : nullptr};
    for (int i = 0; i < 3; ++i)
        if (rows[i] != nullptr) p.tiles[i] = c.take((1 + p.capacity(*rows[i])) * (int64_t)sizeof(TgTileRow));
    p.total = c.total();
    return p;
}

// The jobs before the products.
struct Preps {
    MoePrepList list{};
    bool seek = false;  // no lists of tile rows
    MoePrep &add(MoePrepKind kind) {
        MoePrep &j = list.job[list.n++];
        j.kind = kind;
        return j;
    }
    void place(Weight &w, int64_t ld, int64_t group, int64_t experts, int64_t rows, int64_t cols, char *ws) {
        if (!w.copy) return;
        MoePrep &j = add(kMoeCopy);
        j.src = w.p;
        j.ld = ld;
        j.group_rows = rows;
        j.group_stride = group;
        j.rows = experts * rows;
        j.cols = cols;
        w.p = j.dst = reinterpret_cast<uint16_t *>(ws + w.at);
    }
    void tiles(TgLaunch &L, size_t at, int64_t capacity, char *ws) {
        L.offsets = list.offsets;
        L.order = list.order;
        L.set_top(list.top);
        if (seek) return;
        MoePrep &j = add(kMoeTiles);
        j.height = tile_height(L.tile);
        j.capacity = (int32_t)capacity;
        j.tiles = reinterpret_cast<TgTileRow *>(ws + at);
        L.tile_row = j.tiles;
    }
    void items(TgLaunch &L, size_t at, size_t joins, char *ws) {
        MoePrep &j = add(kMoeItems);
        j.height = L.part_rows;
        j.tiles = reinterpret_cast<TgItem *>(ws + at);
        j.joins = reinterpret_cast<TgItem *>(ws + joins);
        L.items = j.tiles;
        L.joins = j.joins;
    }
    void place(Rows &r, int64_t cols, char *ws) {
        if (!r.copy) return;
        MoePrep &j = add(kMoeGather);
        j.src = r.p;
        j.ld = r.ld;
        j.cols = cols;
        r.slots = j.dst = reinterpret_cast<uint16_t *>(ws + r.at);
    }
};

bool group_ok(int64_t group, int64_t ld, int64_t rows, int64_t cols) {
    return group >= (rows - 1) * ld + cols && group <= ((int64_t)1 << 44);
}

}  // namespace
}  // namespace zopt

using namespace zopt;

ZOPT_EXPORT zopt_status zopt_moe_route(int64_t T, int32_t experts, int32_t top, const void *logits, int64_t ld,
                                       int32_t bf16, int32_t score, const float *bias, int32_t groups,
                                       int32_t top_groups, int32_t renormalise, float scale, int32_t *chosen,
                                       float *weights, int32_t *offsets, int32_t *order, int32_t *place,
                                       void *workspace, size_t *workspace_bytes, void *stream) {
    if (workspace_bytes == nullptr) return ZOPT_ERR_NULL;
    const zopt_status st = check_route(T, experts, top);
    if (st != ZOPT_OK) return st;
    if (!stride_ok(ld, experts) || !range(groups, 1, kMaxRanges < experts ? kMaxRanges : experts) || experts % groups ||
        !range(top_groups, 1, groups) || top > experts / groups * top_groups)
        return ZOPT_ERR_SIZE;
    const bool scored = bias != nullptr || groups > 1;
    const int32_t each = route_block_tokens(T, experts, groups, top, scored);
    const size_t need = plan_bytes(T, experts, each);
    if (workspace == nullptr) {
        *workspace_bytes = need;
        return ZOPT_OK;
    }
    if (offsets == nullptr) return ZOPT_ERR_NULL;
    if (T > 0 && (logits == nullptr || chosen == nullptr || weights == nullptr || order == nullptr || place == nullptr))
        return ZOPT_ERR_NULL;
    if ((bf16 != 0 && bf16 != 1) || (score != ZOPT_SCORE_SOFTMAX && score != ZOPT_SCORE_SIGMOID) ||
        (renormalise != 0 && renormalise != 1) || !std::isfinite(scale))
        return ZOPT_ERR_HYPER;
    const zopt_status ws = workspace_check(need, workspace, *workspace_bytes);
    if (ws != ZOPT_OK) return ws;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const PlanArgs p = plan_args(T, experts, top, each, chosen, workspace, offsets, order, place);
    if (T == 0) return device(launch_plan(p, s));
    const RouteArgs a{T, experts, top, bf16, score == ZOPT_SCORE_SIGMOID, groups, top_groups, renormalise, scale, logits,
                      ld, bias, chosen, weights, p.block_tokens, 0, 0, scored};
    return device(launch_route(a, p, s));
}

ZOPT_EXPORT zopt_status zopt_moe_plan(int64_t T, int32_t experts, int32_t top, const int32_t *chosen, int32_t *offsets,
                                      int32_t *order, int32_t *place, void *workspace, size_t *workspace_bytes,
                                      void *stream) {
    if (workspace_bytes == nullptr) return ZOPT_ERR_NULL;
    // (any number of experts a token, the same one more than once too)
    if (!range(T, 0, kMaxRows) || !range(experts, 1, kMaxExperts) || !range(top, 1, kMaxTop) || T * top > kMaxSlots)
        return ZOPT_ERR_SIZE;
    const int32_t each = route_block_tokens(T, -experts, 1, top, false);
    const size_t need = plan_bytes(T, experts, each);
    if (workspace == nullptr) {
        *workspace_bytes = need;
        return ZOPT_OK;
    }
    if (offsets == nullptr || (T > 0 && (chosen == nullptr || order == nullptr || place == nullptr)))
        return ZOPT_ERR_NULL;
    const zopt_status ws = workspace_check(need, workspace, *workspace_bytes);
    if (ws != ZOPT_OK) return ws;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const PlanArgs p = plan_args(T, experts, top, each, chosen, workspace, offsets, order, place);
    if (T > 0) ZOPT_TRY(launch_plan_count(p, s));
    return device(launch_plan(p, s));
}

ZOPT_EXPORT zopt_status zopt_moe_route_backward(int64_t T, int32_t experts, int32_t top, const float *dweights,
                                                const void *logits, int64_t ld, int32_t bf16, int32_t score,
                                                int32_t renormalise, float scale, const int32_t *chosen, void *dlogits,
                                                int64_t lddl, void *stream) {
    const zopt_status st = check_route(T, experts, top);
    if (st != ZOPT_OK) return st;
    if (!stride_ok(ld, experts) || !stride_ok(lddl, experts)) return ZOPT_ERR_SIZE;
    if ((bf16 != 0 && bf16 != 1) || (score != ZOPT_SCORE_SOFTMAX && score != ZOPT_SCORE_SIGMOID) ||
        (renormalise != 0 && renormalise != 1) || !std::isfinite(scale))
        return ZOPT_ERR_HYPER;
    if (T == 0) return ZOPT_OK;
    if (dweights == nullptr || logits == nullptr || chosen == nullptr || dlogits == nullptr) return ZOPT_ERR_NULL;
    const RouteBackArgs a{T, experts, top, bf16, score == ZOPT_SCORE_SIGMOID, renormalise, scale, logits, ld, chosen,
                          dweights, dlogits, lddl};
    return device(launch_route_back(a, static_cast<hipStream_t>(stream)));
}

namespace {

zopt_status check_moe(int64_t T, int64_t D, int64_t F, int32_t E, int32_t k, int64_t ldx, int64_t ldw, int64_t groupw,
                      int64_t ldd, int64_t groupd) {
    if (!range(T, 0, kMaxRows) || !range(D, 1, kMaxSide) || !range(F, 1, kMaxSide)) return ZOPT_ERR_SIZE;
    if (!range(E, 1, kMaxExperts) || !range(k, 1, kMaxTop) || T * k > kMaxSlots) return ZOPT_ERR_SIZE;
    if (!stride_ok(ldx, D) || !stride_ok(ldw, D) || !stride_ok(ldd, F)) return ZOPT_ERR_SIZE;
    if (!group_ok(groupw, ldw, F, D) || !group_ok(groupd, ldd, D, F)) return ZOPT_ERR_SIZE;
    return ZOPT_OK;
}

}  // namespace

ZOPT_EXPORT zopt_status zopt_moe_forward(int64_t T, int64_t D, int64_t F, int32_t experts, int32_t top,
                                         const uint16_t *x, int64_t ldx, const uint16_t *w_gate, const uint16_t *w_up,
                                         int64_t ldw, int64_t w_expert, const uint16_t *w_down, int64_t ldd,
                                         int64_t wd_expert, int32_t act, const float *weights, const int32_t *offsets,
                                         const int32_t *order, const int32_t *place, uint16_t *y, int64_t ldy,
                                         void *workspace, size_t *workspace_bytes, void *stream) {
    if (workspace_bytes == nullptr) return ZOPT_ERR_NULL;
    const zopt_status st = check_moe(T, D, F, experts, top, ldx, ldw, w_expert, ldd, wd_expert);
    if (st != ZOPT_OK) return st;
    if (!stride_ok(ldy, D)) return ZOPT_ERR_SIZE;
    MoePlan p = moe_plan(T, D, F, experts, top, x, ldx, nullptr, 0, w_gate, w_up, ldw, w_expert, w_down, ldd, wd_expert,
                         false);
    if (workspace == nullptr) {
        *workspace_bytes = p.total;
        return ZOPT_OK;
    }
    if (w_gate == nullptr || w_up == nullptr || w_down == nullptr || offsets == nullptr) return ZOPT_ERR_NULL;
    if (T > 0 && (x == nullptr || y == nullptr || weights == nullptr || order == nullptr || place == nullptr))
        return ZOPT_ERR_NULL;
    if (act != kActSilu && act != kActGelu) return ZOPT_ERR_HYPER;
    const zopt_status ok = workspace_check(p.total, workspace, *workspace_bytes);
    if (ok != ZOPT_OK) return ok;
    if (T == 0) return ZOPT_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    Preps preps;
    preps.list.experts = experts;
    preps.list.top = top;
    preps.list.slots = p.S;
    preps.list.offsets = offsets;
    preps.list.order = order;
    // Where that is all there is to prepare, the products find few groups' tile rows
    // themselves, 1 us each: 48 tokens' pass over 16 experts of 768 x 512 takes 28 us
    // on the GPU, 32 with a launch for the lists.
    preps.seek = experts <= 64 && tile_seeks(p.glu.tile) && tile_seeks(p.down.tile) && !p.wg.copy && !p.wu.copy &&
                 !p.wd.copy && !p.x.copy;
    preps.tiles(p.glu, p.tiles[0], p.capacity(p.glu), ws);
    preps.tiles(p.down, p.tiles[1], p.capacity(p.down), ws);
    preps.place(p.wg, ldw, w_expert, experts, F, D, ws);
    preps.place(p.wu, ldw, w_expert, experts, F, D, ws);
    preps.place(p.wd, ldd, wd_expert, experts, D, F, ws);
    preps.place(p.x, D, ws);
    ZOPT_TRY(launch_moe_prep(preps.list, s));
    const TgOperand xs = p.rows_along(p.x, D);
    p.glu.prob[0].nseg = 2;
    p.glu.prob[0].seg[0] = MoePlan::segment(xs, MoePlan::along(p.wg, F, D));
    p.glu.prob[0].seg[1] = MoePlan::segment(xs, MoePlan::along(p.wu, F, D));
    p.glu.group_stride = p.wg.group;
    p.glu.act = act;
    p.glu.h = reinterpret_cast<uint16_t *>(ws + p.h);
    p.glu.ldc = p.Fp;
    ZOPT_TRY(launch_rows_glu(p.x.gathered, p.glu, s));
    p.down.prob[0].seg[0] = MoePlan::segment(p.slots_along(ws + p.h, p.Fp, F), MoePlan::along(p.wd, D, F));
    p.down.prob[0].out = reinterpret_cast<uint16_t *>(ws + p.rows);
    p.down.row_scale = reinterpret_cast<uint8_t *>(ws + p.scale);
    p.down.ldscale = p.scales;
    p.down.ldc = p.Dp;
    p.down.group_stride = p.wd.group;
    ZOPT_TRY(launch_rows(false, p.down, s));
    MoeCombine c{};
    c.tokens = T;
    c.cols = D;
    c.top = top;
    c.slots = p.S;
    c.place = place;
    c.weights = weights;
    c.rows = reinterpret_cast<const uint16_t *>(ws + p.rows);
    c.scale = reinterpret_cast<const uint8_t *>(ws + p.scale);
    c.ldscale = p.scales;
    c.ld = p.Dp;
    c.out = y;
    c.ldo = ldy;
    return device(launch_moe_combine(c, s));
}

ZOPT_EXPORT zopt_status zopt_moe_backward(int64_t T, int64_t D, int64_t F, int32_t experts, int32_t top,
                                          const uint16_t *dy, int64_t lddy, const uint16_t *x, int64_t ldx,
                                          const uint16_t *w_gate, const uint16_t *w_up, int64_t ldw, int64_t w_expert,
                                          const uint16_t *w_down, int64_t ldd, int64_t wd_expert, int32_t act,
                                          const float *weights, const int32_t *offsets, const int32_t *order,
                                          const int32_t *place, uint16_t *dx, int64_t lddx, uint16_t *dw_gate,
                                          uint16_t *dw_up, int64_t lddw, int64_t dw_expert, uint16_t *dw_down,
                                          int64_t lddd, int64_t dwd_expert, float *dweights, void *workspace,
                                          size_t *workspace_bytes, void *stream) {
    if (workspace_bytes == nullptr) return ZOPT_ERR_NULL;
    const zopt_status st = check_moe(T, D, F, experts, top, ldx, ldw, w_expert, ldd, wd_expert);
    if (st != ZOPT_OK) return st;
    if (!stride_ok(lddy, D) || !stride_ok(lddx, D) || !stride_ok(lddw, D) || !stride_ok(lddd, F)) return ZOPT_ERR_SIZE;
    if (!group_ok(dw_expert, lddw, F, D) || !group_ok(dwd_expert, lddd, D, F)) return ZOPT_ERR_SIZE;
    MoePlan p = moe_plan(T, D, F, experts, top, x, ldx, dy, lddy, w_gate, w_up, ldw, w_expert, w_down, ldd, wd_expert,
                         true);
    if (workspace == nullptr) {
        *workspace_bytes = p.total;
        return ZOPT_OK;
    }
    if (w_gate == nullptr || w_up == nullptr || w_down == nullptr || offsets == nullptr || dw_gate == nullptr ||
        dw_up == nullptr || dw_down == nullptr)
        return ZOPT_ERR_NULL;
    if (T > 0 && (dy == nullptr || x == nullptr || weights == nullptr || order == nullptr || place == nullptr ||
                  dx == nullptr || dweights == nullptr))
        return ZOPT_ERR_NULL;
    if (act != kActSilu && act != kActGelu) return ZOPT_ERR_HYPER;
    const zopt_status ok = workspace_check(p.total, workspace, *workspace_bytes);
    if (ok != ZOPT_OK) return ok;
    hipStream_t s = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    if (T == 0) {
        ZOPT_TRY(launch_fill_zero_groups(dw_gate, lddw, dw_expert, experts, F, D, s));
        ZOPT_TRY(launch_fill_zero_groups(dw_up, lddw, dw_expert, experts, F, D, s));
        return device(launch_fill_zero_groups(dw_down, lddd, dwd_expert, experts, D, F, s));
    }
    Preps preps;
    preps.list.experts = experts;
    preps.list.top = top;
    preps.list.slots = p.S;
    preps.list.offsets = offsets;
    preps.list.order = order;
    preps.tiles(p.glu, p.tiles[0], p.capacity(p.glu), ws);
    preps.tiles(p.dhf, p.tiles[1], p.capacity(p.dhf), ws);
    preps.tiles(p.dx, p.tiles[2], p.capacity(p.dx), ws);
    preps.items(p.dwgu, p.items[0], p.joins[0], ws);
    preps.items(p.dwd, p.items[1], p.joins[1], ws);
    preps.place(p.wg, ldw, w_expert, experts, F, D, ws);
    preps.place(p.wu, ldw, w_expert, experts, F, D, ws);
    preps.place(p.wd, ldd, wd_expert, experts, D, F, ws);
    preps.place(p.x, D, ws);
    preps.place(p.dy, D, ws);
    MoePrep &j = preps.add(kMoeShares);
    j.weights = weights;
    j.share = reinterpret_cast<float *>(ws + p.share);
    ZOPT_TRY(launch_moe_prep(preps.list, s));
    // dh = dy w_down, before the slots' weights
    p.dhf.prob[0].seg[0] = MoePlan::segment(p.rows_along(p.dy, D), MoePlan::across(p.wd, D, F));
    p.dhf.prob[0].sum = reinterpret_cast<float *>(ws + p.dh);
    p.dhf.ldsum = p.Fp;
    p.dhf.group_stride = p.wd.group;
    ZOPT_TRY(launch_rows_float(p.dy.gathered, p.dhf, s));
    // g and u again; dg, du, share h and the dots
    const TgOperand xs = p.rows_along(p.x, D);
    p.glu.prob[0].nseg = 2;
    p.glu.prob[0].seg[0] = MoePlan::segment(xs, MoePlan::along(p.wg, F, D));
    p.glu.prob[0].seg[1] = MoePlan::segment(xs, MoePlan::along(p.wu, F, D));
    p.glu.group_stride = p.wg.group;
    p.glu.act = act;
    p.glu.h = reinterpret_cast<uint16_t *>(ws + p.h);
    p.glu.ldc = p.Fp;
    p.glu.dg = reinterpret_cast<uint16_t *>(ws + p.dg);
    p.glu.du = reinterpret_cast<uint16_t *>(ws + p.du);
    p.glu.lddg = p.Fp;
    p.glu.dhf = reinterpret_cast<const float *>(ws + p.dh);
    p.glu.lddh = p.Fp;
    p.glu.share = reinterpret_cast<const float *>(ws + p.share);
    p.glu.dot = reinterpret_cast<float *>(ws + p.dot);
    p.glu.lddot = p.parts;
    ZOPT_TRY(launch_rows_back(p.x.gathered, p.glu, s));
    // dx = dg w_gate + du w_up, a row a slot, then summed over each token's
    p.dx.prob[0].seg[0] = MoePlan::segment(p.slots_along(ws + p.dg, p.Fp, F), MoePlan::across(p.wg, F, D));
    p.dx.prob[0].seg[1] = MoePlan::segment(p.slots_along(ws + p.du, p.Fp, F), MoePlan::across(p.wu, F, D));
    p.dx.prob[0].out = reinterpret_cast<uint16_t *>(ws + p.rows);
    p.dx.row_scale = reinterpret_cast<uint8_t *>(ws + p.scale);
    p.dx.ldscale = p.scales;
    p.dx.ldc = p.Dp;
    p.dx.group_stride = p.wg.group;
    ZOPT_TRY(launch_rows(true, p.dx, s));
    MoeCombine c{};
    c.tokens = T;
    c.cols = D;
    c.top = top;
    c.slots = p.S;
    c.place = place;
    c.rows = reinterpret_cast<const uint16_t *>(ws + p.rows);
    c.scale = reinterpret_cast<const uint8_t *>(ws + p.scale);
    c.ldscale = p.scales;
    c.ld = p.Dp;
    c.out = dx;
    c.ldo = lddx;
    c.dot = reinterpret_cast<const float *>(ws + p.dot);
    c.lddot = p.parts;
    c.parts = (int32_t)p.parts;
    c.dweights = dweights;
    // the weights' gradients
    p.dwgu.part = reinterpret_cast<float *>(ws + p.part[0]);
    p.dwd.part = reinterpret_cast<float *>(ws + p.part[1]);
    const TgOperand xa = p.slots_across(p.x.slots, p.Dp, D);
    p.dwgu.prob[0].seg[0].a = p.slots_across(ws + p.dg, p.Fp, F);
    p.dwgu.prob[0].seg[0].b = xa;
    p.dwgu.prob[1].nseg = 1;
    p.dwgu.prob[1].seg[0].a = p.slots_across(ws + p.du, p.Fp, F);
    p.dwgu.prob[1].seg[0].b = xa;
    p.dwgu.prob[0].out = dw_gate;
    p.dwgu.prob[1].out = dw_up;
    p.dwgu.ldc = lddw;
    p.dwgu.group_out = dw_expert;
    ZOPT_TRY(launch_depth(p.dwgu, s));
    p.dwd.prob[0].seg[0].a = p.slots_across(p.dy.slots, p.Dp, D);
    p.dwd.prob[0].seg[0].b = p.slots_across(ws + p.h, p.Fp, F);
    p.dwd.prob[0].out = dw_down;
    p.dwd.ldc = lddd;
    p.dwd.group_out = dwd_expert;
    ZOPT_TRY(launch_depth(p.dwd, s));
    int i = 0;
    for (const TgLaunch *L : {&p.dwgu, &p.dwd}) {
        MoeJoin &j = c.join[i++];
        j.L = *L;
        tile_shape(L->tile, j.height, j.width, j.rows, j.cols);
    }
    return device(launch_moe_combine(c, s));
}
