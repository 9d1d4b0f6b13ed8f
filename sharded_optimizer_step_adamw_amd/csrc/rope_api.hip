// rope_api.hip -- the C-ABI entry points of the norms and rotation of queries
// and keys (declared in zopt.h).
#include <cmath>

#include "rope_internal.h"
#include "train_api.h"

namespace zopt {
namespace {

constexpr int32_t kMaxHeads = 1 << 16;
constexpr int64_t kMaxHeadStride = (int64_t)1 << 40;

// Strides that only reads go by
bool reads_ok(int64_t token, int64_t head) { return range(token, 0, kMaxHeadStride) && range(head, 0, kMaxHeadStride); }
// ... and of an output, whose rows must not overlap: tokens of heads, or heads of tokens
bool writes_ok(int64_t T, int64_t heads, int64_t width, int64_t token, int64_t head) {
    if (!reads_ok(token, head)) return false;
    const int64_t t = T > 1 ? token : kMaxHeadStride, h = heads > 1 ? head : kMaxHeadStride;
    if (T <= 1 || heads <= 1) return t >= width && h >= width;
    return (h >= width && t >= (heads - 1) * h + width) || (t >= width && h >= (T - 1) * t + width);
}

zopt_status check_sizes(int64_t T, int32_t hq, int32_t hk, int32_t width, int32_t rot, int64_t positions) {
    if (!range(T, 0, kMaxRows) || !range(hq, 1, kMaxHeads) || !range(hk, 0, kMaxHeads)) return ZOPT_ERR_SIZE;
    if (!range(width, 1, kMaxHeadWidth) || !range(rot, 0, width) || (rot & 1)) return ZOPT_ERR_SIZE;
    if (!range(positions, 0, kMaxRows)) return ZOPT_ERR_SIZE;
    return ZOPT_OK;
}
bool hyper_ok(float eps, int32_t style) {
    return std::isfinite(eps) && eps >= 0.0f && (style == ZOPT_ROPE_HALF || style == ZOPT_ROPE_PAIRS);
}
RopeArgs common(int64_t T, int32_t hq, int32_t hk, int32_t width, int32_t rot, const float *table, int64_t positions,
                const int64_t *position, float eps, int32_t style) {
    RopeArgs a{};
    a.side[0].heads = hq;
    a.side[1].heads = hk;
    a.tokens = T;
    a.positions = rot > 0 ? positions : INT64_MAX;
    a.width = width;
    a.rot = rot;
    a.pairs = style == ZOPT_ROPE_PAIRS;
    a.eps = eps;
    a.table = reinterpret_cast<const float2 *>(table);
    a.position = position;
    return a;
}

}  // namespace
}  // namespace zopt

using namespace zopt;

ZOPT_EXPORT zopt_status zopt_rope_table(int64_t positions, int32_t rot, double base, float *table, void *stream) {
    if (!range(positions, 0, kMaxRows) || !range(rot, 2, kMaxHeadWidth) || (rot & 1)) return ZOPT_ERR_SIZE;
    if (!std::isfinite(base) || !(base > 0)) return ZOPT_ERR_HYPER;
    if (positions == 0) return ZOPT_OK;
    if (table == nullptr) return ZOPT_ERR_NULL;
    return device(launch_rope_table(positions, rot, base, reinterpret_cast<float2 *>(table),
                                    static_cast<hipStream_t>(stream)));
}

ZOPT_EXPORT zopt_status zopt_qk_norm_rope(int64_t T, int32_t heads_q, int32_t heads_k, int32_t width, int32_t rot,
                                          const uint16_t *q, int64_t q_token, int64_t q_head, const uint16_t *k,
                                          int64_t k_token, int64_t k_head, const float *table, int64_t positions,
                                          const int64_t *position, const uint16_t *w_q, const uint16_t *w_k, float eps,
                                          int32_t style, uint16_t *yq, int64_t yq_token, int64_t yq_head, uint16_t *yk,
                                          int64_t yk_token, int64_t yk_head, void *stream) {
    const zopt_status st = check_sizes(T, heads_q, heads_k, width, rot, positions);
    if (st != ZOPT_OK) return st;
    if (!reads_ok(q_token, q_head) || !writes_ok(T, heads_q, width, yq_token, yq_head)) return ZOPT_ERR_SIZE;
    if (heads_k > 0 && (!reads_ok(k_token, k_head) || !writes_ok(T, heads_k, width, yk_token, yk_head)))
        return ZOPT_ERR_SIZE;
    if (!hyper_ok(eps, style)) return ZOPT_ERR_HYPER;
    if (T == 0) return ZOPT_OK;
    if (q == nullptr || yq == nullptr || (heads_k > 0 && (k == nullptr || yk == nullptr))) return ZOPT_ERR_NULL;
    if (rot > 0 && positions > 0 && table == nullptr) return ZOPT_ERR_NULL;
    RopeArgs a = common(T, heads_q, heads_k, width, rot, table, positions, position, eps, style);
    a.side[0] = RopeSide{q, nullptr, yq, q_token, q_head, 0, 0, yq_token, yq_head, w_q, nullptr, heads_q};
    a.side[1] = RopeSide{k, nullptr, yk, k_token, k_head, 0, 0, yk_token, yk_head, w_k, nullptr, heads_k};
    plan_rope(a);
    return device(launch_rope(a, static_cast<hipStream_t>(stream)));
}

ZOPT_EXPORT zopt_status zopt_qk_norm_rope_backward(
    int64_t T, int32_t heads_q, int32_t heads_k, int32_t width, int32_t rot, const uint16_t *dyq, int64_t dyq_token,
    int64_t dyq_head, const uint16_t *dyk, int64_t dyk_token, int64_t dyk_head, const uint16_t *q, int64_t q_token,
    int64_t q_head, const uint16_t *k, int64_t k_token, int64_t k_head, const float *table, int64_t positions,
    const int64_t *position, const uint16_t *w_q, const uint16_t *w_k, float eps, int32_t style, uint16_t *dq,
    int64_t dq_token, int64_t dq_head, uint16_t *dk, int64_t dk_token, int64_t dk_head, uint16_t *dw_q, uint16_t *dw_k,
    void *workspace, size_t *workspace_bytes, void *stream) {
    if (workspace_bytes == nullptr) return ZOPT_ERR_NULL;
    const zopt_status st = check_sizes(T, heads_q, heads_k, width, rot, positions);
    if (st != ZOPT_OK) return st;
    if (!reads_ok(dyq_token, dyq_head) || !reads_ok(q_token, q_head) || !writes_ok(T, heads_q, width, dq_token, dq_head))
        return ZOPT_ERR_SIZE;
    if (heads_k > 0 && (!reads_ok(dyk_token, dyk_head) || !reads_ok(k_token, k_head) ||
                        !writes_ok(T, heads_k, width, dk_token, dk_head)))
        return ZOPT_ERR_SIZE;
    RopeArgs a = common(T, heads_q, heads_k, width, rot, table, positions, position, eps, style);
    plan_rope(a);
    const bool sums = dw_q != nullptr || dw_k != nullptr;
    const size_t need = sums ? (size_t)up((int64_t)a.blocks * width * 4, 256) : 0;
    if (workspace == nullptr) {
        *workspace_bytes = need;
        return ZOPT_OK;
    }
    if (!hyper_ok(eps, style)) return ZOPT_ERR_HYPER;
    if (dw_k != nullptr && heads_k == 0) return ZOPT_ERR_NULL;
    if (T > 0) {
        if (dyq == nullptr || q == nullptr || dq == nullptr) return ZOPT_ERR_NULL;
        if (heads_k > 0 && (dyk == nullptr || k == nullptr || dk == nullptr)) return ZOPT_ERR_NULL;
        if (rot > 0 && positions > 0 && table == nullptr) return ZOPT_ERR_NULL;
    }
    const zopt_status ws = workspace_check(need, workspace, *workspace_bytes);
    if (ws != ZOPT_OK) return ws;
    a.side[0] = RopeSide{q, dyq, dq, q_token, q_head, dyq_token, dyq_head, dq_token, dq_head, w_q, dw_q, heads_q};
    a.side[1] = RopeSide{k, dyk, dk, k_token, k_head, dyk_token, dyk_head, dk_token, dk_head, w_k, dw_k, heads_k};
    a.part = reinterpret_cast<float *>(workspace);
    return device(launch_rope_back(a, static_cast<hipStream_t>(stream)));
}
