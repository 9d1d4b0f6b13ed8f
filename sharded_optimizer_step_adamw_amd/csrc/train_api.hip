// train_api.hip -- the C-ABI entry points of the gradient operators (declared
// in zopt.h): linear cross entropy, the gated feed-forward block, 8-bit
// activation checkpoints.
//
// As everywhere in the library, arguments are checked first, the launches are
// planned on the host, and everything is enqueued on the caller's stream
// without synchronising.  Each call's plan is made by one function that both
// the size query and the call itself run, so they cannot disagree.
#include <cmath>

#include "train_internal.h"
#include "zopt.h"

#define ZOPT_EXPORT extern "C" __attribute__((visibility("default")))

namespace zopt {
namespace {

constexpr int64_t kMaxSide = 1 << 21;          // D, F, V: a 256-row panel stays below 2^31 bytes
constexpr int64_t kMaxRows = 1 << 30;          // T
constexpr int64_t kMaxStride = (1 << 22) - 8;  // of an operand read in place
// Exponentials of the logits held at once (2 GiB, under 1% of the 288 GB).
// Rows are taken in as few pieces as that allows, since every piece after the
// first reads and writes the fp32 sums of dW once (8 V D bytes) and reads w
// again: [16384, 4096] x 131072 words takes 42.5 ms in two pieces, half of its rows
// 21.0 in one; [8192, 4096] x 262144 words 43.7 in two, half of its rows 21.3.
constexpr int64_t kPieceBytes = (int64_t)1 << 31;

inline int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// Offsets into a workspace, in order, 256-byte aligned.
struct Carve {
    size_t off = 0;
    size_t take(int64_t bytes) {
        const size_t at = off;
        off += (size_t)up(bytes, 256);
        return at;
    }
    size_t total() const { return off; }
};

// A 16-bit operand [rows, cols] as the products read it: in place if its
// contiguous side, stride and base are multiples of 8 elements, else a padded
// copy in the workspace.
struct Input {
    const uint16_t *p;
    int64_t ld, rows, cols;
    bool copy;
    size_t at;
};
bool in_place(const uint16_t *p, int64_t ld, int64_t cols) {
    return aligned16(p) && !(ld & 7) && !(cols & 7) && ld <= kMaxStride;
}
Input input(const uint16_t *p, int64_t ld, int64_t rows, int64_t cols, bool force, Carve &c) {
    Input in{p, ld, rows, cols, false, 0};
    in.copy = force || !in_place(p, ld, cols);
    if (in.copy) {
        in.ld = up(cols, 8);
        in.at = c.take(rows * in.ld * 2);
    }
    return in;
}
// The jobs before a call's products.
struct Preps {
    TgPrepList list{};
    TgPrep &add(TgPrepKind kind, int64_t rows, int64_t cols) {
        TgPrep &j = list.job[list.n++];
        j.kind = kind;
        j.rows = rows;
        j.cols = cols;
        return j;
    }
    // the padded copy of an operand that needs one, without the rows whose
    // target (if given) is `ignore`
    void place(Input &in, int64_t src_ld, char *ws, const int64_t *target = nullptr, int64_t ignore = 0) {
        if (!in.copy) return;
        TgPrep &j = add(kPrepCopy, in.rows, in.cols);
        j.src = in.p;
        j.ld = src_ld;
        j.target = target;
        j.ignore = ignore;
        in.p = j.dst = reinterpret_cast<uint16_t *>(ws + in.at);
    }
    // an operand from its checkpoint
    void unpack(Input &in, const uint8_t *q, const uint8_t *scale, char *ws) {
        TgPrep &j = add(kPrepUnpack, in.rows, in.cols);
        j.q = q;
        j.scale = scale;
        in.p = j.dst = reinterpret_cast<uint16_t *>(ws + in.at);
    }
    hipError_t run(hipStream_t s) { return launch_prep(list, s); }
};
// rows [r0, r0 + n) of an operand that the reduction runs along (outer: rows)
TgOperand along(const Input &in, int64_t r0, int64_t n) {
    return TgOperand{in.p + r0 * in.ld, in.ld, (int32_t)n, (int32_t)up(in.cols, 8)};
}
// ... and across (reduction over the rows)
TgOperand across(const Input &in, int64_t r0, int64_t n) {
    return TgOperand{in.p + r0 * in.ld, in.ld, (int32_t)up(in.cols, 8), (int32_t)n};
}
TgSegment segment(const TgOperand &a, const TgOperand &b) {
    const int32_t k = a.k > b.k ? a.k : b.k;
    return TgSegment{a, b, (k + 63) / 64 * 2};
}

// A product's launch over one or two problems of the same sizes.
struct Product {
    TgLaunch L{};
    Product(TgEpilogue epi, int64_t M, int64_t N, const TgSegment &s0, const TgSegment *s1 = nullptr) : epi(epi) {
        L.nprob = 1;
        L.M = (int32_t)M;
        L.N = (int32_t)N;
        L.prob[0].seg[0] = s0;
        L.prob[0].nseg = s1 ? 2 : 1;
        if (s1) L.prob[0].seg[1] = *s1;
    }
    void second(const TgSegment &s) {
        L.prob[1].seg[0] = s;
        L.prob[1].nseg = 1;
        L.nprob = 2;
    }
    // scratch for the parts of a split reduction
    size_t parts() {
        plan_tg(epi, L);
        return tg_part_bytes(epi, L);
    }
    hipError_t run(bool a_km, bool b_km, char *part, hipStream_t s) {
        plan_tg(epi, L);
        L.part = reinterpret_cast<float *>(part);
        return launch_tg(epi, a_km, b_km, L, s);
    }

   private:
    TgEpilogue epi;
};
inline size_t larger(size_t a, size_t b) { return a > b ? a : b; }

bool range(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }
bool stride_ok(int64_t ld, int64_t cols) { return ld >= cols && ld <= ((int64_t)1 << 31); }

zopt_status device(hipError_t e) { return e == hipSuccess ? ZOPT_OK : ZOPT_ERR_DEVICE; }
#define ZOPT_TRY(x)                                 \
    do {                                            \
        const hipError_t e_ = (x);                  \
        if (e_ != hipSuccess) return ZOPT_ERR_DEVICE; \
    } while (0)

zopt_status workspace_check(size_t need, void *workspace, size_t given) {
    if (given < need || ((uintptr_t)workspace & 255)) return ZOPT_ERR_WORKSPACE;
    return ZOPT_OK;
}

// ------------------------------------------------------- cross entropy plan

struct XentPlan {
    Input x, w;
    int64_t piece;   // rows of a piece
    int32_t pieces, groups;
    int64_t lde;     // row stride of the exponentials
    size_t e, stats, zt, row, factor, sum, part, total;
    Input probs(char *ws, int64_t n) const {
        return Input{reinterpret_cast<const uint16_t *>(ws + e), lde, n, w.rows, false, 0};
    }
    Product logits(int64_t r0, int64_t n) const {
        return Product(kTgXent, n, w.rows, segment(along(x, r0, n), along(w, 0, w.rows)));
    }
    Product dx(char *ws, int64_t n) const {
        return Product(kTgStore, n, w.cols, segment(along(probs(ws, n), 0, n), across(w, 0, w.rows)));
    }
    Product dw(char *ws, int64_t r0, int64_t n) const {
        Product p(pieces > 1 ? kTgSum : kTgStore, w.rows, w.cols,
                  segment(across(probs(ws, n), 0, n), across(x, r0, n)));
        p.L.sum_in = r0 > 0;
        p.L.sum_out = r0 + n < x.rows;
        return p;
    }
};
XentPlan xent_plan(int64_t T, int64_t D, int64_t V, const uint16_t *x, int64_t ldx, const uint16_t *w, int64_t ldw,
                   bool dx, bool dw) {
    XentPlan p{};
    Carve c;
    // (dW sums over rows: an ignored row must not reach it, whatever it holds)
    p.x = input(x, ldx, T, D, dw, c);
    p.w = input(w, ldw, V, D, false, c);
    p.lde = up(V, 64);
    p.groups = (int32_t)((V + kXentGroup - 1) / kXentGroup);
    int64_t most = kPieceBytes / (2 * p.lde) / 256 * 256;
    if (most < 256) most = 256;
    p.pieces = (int32_t)((T + most - 1) / most);
    if (p.pieces < 1) p.pieces = 1;
    p.piece = up((T + p.pieces - 1) / p.pieces, 256);
    if (p.piece > T) p.piece = T;
    if (dx || dw) p.e = c.take(p.piece * p.lde * 2);
    p.stats = c.take(p.piece * p.groups * (int64_t)sizeof(float2));
    p.zt = c.take(p.piece * 4);
    p.row = c.take(T * 4);
    p.factor = c.take(4);
    if (dw && p.pieces > 1) p.sum = c.take(V * up(D, 4) * 4);
    size_t parts = 0;
    for (int32_t k = 0; k < p.pieces; ++k) {
        const int64_t r0 = k * p.piece, n = T - r0 < p.piece ? T - r0 : p.piece;
        if (n <= 0) break;
        if (k > 0 && r0 + n < T) continue;  // (pieces between are as the first)
        parts = larger(parts, p.logits(r0, n).parts());
        if (dx) parts = larger(parts, p.dx(nullptr, n).parts());
        if (dw) parts = larger(parts, p.dw(nullptr, r0, n).parts());
    }
    p.part = c.take(parts);
    p.total = c.total();
    return p;
}

// ------------------------------------------------------------ gated block plan

struct GluPlan {
    Input x, wg, wu;
    int64_t fp;      // row stride of dg and du
    size_t dg, du, part, total;
    Input grad(char *ws, size_t at) const {
        return Input{reinterpret_cast<const uint16_t *>(ws + at), fp, x.rows, wg.rows, false, 0};
    }
    Product products(TgEpilogue epi) const {
        const TgSegment up = segment(along(x, 0, x.rows), along(wu, 0, wu.rows));
        return Product(epi, x.rows, wg.rows, segment(along(x, 0, x.rows), along(wg, 0, wg.rows)), &up);
    }
    Product dx(char *ws) const {
        const TgSegment up = segment(along(grad(ws, du), 0, x.rows), across(wu, 0, wu.rows));
        return Product(kTgStore, x.rows, x.cols,
                       segment(along(grad(ws, dg), 0, x.rows), across(wg, 0, wg.rows)), &up);
    }
    Product dw(char *ws) const {
        Product p(kTgStore, wg.rows, x.cols, segment(across(grad(ws, dg), 0, x.rows), across(x, 0, x.rows)));
        p.second(segment(across(grad(ws, du), 0, x.rows), across(x, 0, x.rows)));
        return p;
    }
};
GluPlan glu_plan(int64_t T, int64_t D, int64_t F, const uint16_t *x, int64_t ldx, const uint8_t *x8,
                 const uint16_t *wg, const uint16_t *wu, int64_t ldw, bool back) {
    GluPlan p{};
    Carve c;
    p.x = input(x, ldx, T, D, x8 != nullptr, c);
    // (the products take both with one row stride)
    const bool copy = !in_place(wg, ldw, D) || !in_place(wu, ldw, D);
    p.wg = input(wg, ldw, F, D, copy, c);
    p.wu = input(wu, ldw, F, D, copy, c);
    p.fp = up(F, 8);
    if (back) {
        p.dg = c.take(T * p.fp * 2);
        p.du = c.take(T * p.fp * 2);
    }
    if (T > 0) {
        size_t parts = p.products(back ? kTgGluBack : kTgGlu).parts();
        if (back) parts = larger(parts, larger(p.dx(nullptr).parts(), p.dw(nullptr).parts()));
        p.part = c.take(parts);
    }
    p.total = c.total();
    return p;
}

}  // namespace
}  // namespace zopt

using namespace zopt;

ZOPT_EXPORT zopt_status zopt_linear_xent(int64_t T, int64_t D, int64_t V, const uint16_t *x, int64_t ldx,
                                         const uint16_t *w, int64_t ldw, const int64_t *target, int64_t ignore_index,
                                         int32_t mean, float grad_scale, float *loss, float *row_loss, uint16_t *dx,
                                         int64_t lddx, uint16_t *dw, int64_t lddw, void *workspace,
                                         size_t *workspace_bytes, void *stream) {
    if (workspace_bytes == nullptr) return ZOPT_ERR_NULL;
    if (!range(T, 0, kMaxRows) || !range(D, 1, kMaxSide) || !range(V, 1, kMaxSide)) return ZOPT_ERR_SIZE;
    if (!stride_ok(ldx, D) || !stride_ok(ldw, D)) return ZOPT_ERR_SIZE;
    if ((dx != nullptr && !stride_ok(lddx, D)) || (dw != nullptr && !stride_ok(lddw, D))) return ZOPT_ERR_SIZE;
    XentPlan p = xent_plan(T, D, V, x, ldx, w, ldw, dx != nullptr, dw != nullptr);
    if (workspace == nullptr) {
        *workspace_bytes = p.total;
        return ZOPT_OK;
    }
    if (w == nullptr || loss == nullptr || (T > 0 && (x == nullptr || target == nullptr))) return ZOPT_ERR_NULL;
    if ((mean != 0 && mean != 1) || !std::isfinite(grad_scale)) return ZOPT_ERR_HYPER;
    const zopt_status st = workspace_check(p.total, workspace, *workspace_bytes);
    if (st != ZOPT_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    float *factor = reinterpret_cast<float *>(ws + p.factor);
    float *row = row_loss != nullptr ? row_loss : reinterpret_cast<float *>(ws + p.row);
    if (T == 0) {
        ZOPT_TRY(launch_xent_total(TgTotal{row, target, 0, ignore_index, mean, loss}, s));
        if (dw != nullptr) ZOPT_TRY(launch_fill_zero(dw, lddw, V, D, s));
        return ZOPT_OK;
    }
    Preps preps;
    if (dx != nullptr || dw != nullptr) {
        TgPrep &j = preps.add(kPrepCount, T, 0);
        j.target = target;
        j.ignore = ignore_index;
        j.mean = mean;
        j.grad_scale = grad_scale;
        j.factor = factor;
    }
    preps.place(p.x, ldx, ws, dw != nullptr ? target : nullptr, ignore_index);
    preps.place(p.w, ldw, ws);
    ZOPT_TRY(preps.run(s));
    uint16_t *e = dx != nullptr || dw != nullptr ? reinterpret_cast<uint16_t *>(ws + p.e) : nullptr;
    float2 *stats = reinterpret_cast<float2 *>(ws + p.stats);
    float *zt = reinterpret_cast<float *>(ws + p.zt);
    const TgTotal total{row, target, T, ignore_index, mean, loss};
    // Exponentials beyond twice the memory-side cache go past the caches: for
    // [8192, 768] x 50304 (824 MB) the pass that turns them into probabilities
    // takes 320 us so and 372 otherwise, the product after it 528 and 556, the one
    // that makes them 682 and 685.
    const int32_t past = p.piece * p.lde * 2 > 2 * kCacheBytes;
    for (int32_t k = 0; k < p.pieces; ++k) {
        const int64_t r0 = k * p.piece, n = T - r0 < p.piece ? T - r0 : p.piece;
        if (n <= 0) break;
        Product logits = p.logits(r0, n);
        TgLaunch &L = logits.L;
        L.e = e;
        L.lde = e != nullptr ? p.lde : 0;
        L.past = past;
        L.stats = stats;
        L.ldstat = p.groups;
        L.target = target + r0;
        L.zt = zt;
        ZOPT_TRY(logits.run(false, false, ws + p.part, s));
        ZOPT_TRY(launch_xent_rows(stats, p.groups, target + r0, ignore_index, (int32_t)V, zt, n, row + r0, e, p.lde, past,
                                  s));
        // (the last product's launch also forms the loss)
        const bool last = r0 + n == T;
        if (dx != nullptr) {
            Product g = p.dx(ws, n);
            g.L.prob[0].out = dx + r0 * lddx;
            g.L.ldc = lddx;
            g.L.alpha = factor;
            if (last && dw == nullptr) g.L.sum_up = total;
            ZOPT_TRY(g.run(false, true, ws + p.part, s));
        }
        if (dw != nullptr) {
            Product g = p.dw(ws, r0, n);
            g.L.prob[0].out = dw;
            g.L.prob[0].sum = reinterpret_cast<float *>(ws + p.sum);
            g.L.ldc = lddw;
            g.L.alpha = factor;
            if (last) g.L.sum_up = total;
            ZOPT_TRY(g.run(true, true, ws + p.part, s));
        }
    }
    if (e == nullptr) ZOPT_TRY(launch_xent_total(total, s));
    return ZOPT_OK;
}

ZOPT_EXPORT zopt_status zopt_glu_forward(int64_t T, int64_t D, int64_t F, const uint16_t *x, int64_t ldx,
                                         const uint16_t *w_gate, const uint16_t *w_up, int64_t ldw, int32_t act,
                                         uint16_t *h, int64_t ldh, uint8_t *g8, uint8_t *g_scale, uint8_t *u8,
                                         uint8_t *u_scale, void *workspace, size_t *workspace_bytes, void *stream) {
    if (workspace_bytes == nullptr) return ZOPT_ERR_NULL;
    if (!range(T, 0, kMaxRows) || !range(D, 1, kMaxSide) || !range(F, 1, kMaxSide)) return ZOPT_ERR_SIZE;
    if (!stride_ok(ldx, D) || !stride_ok(ldw, D) || !stride_ok(ldh, F)) return ZOPT_ERR_SIZE;
    GluPlan p = glu_plan(T, D, F, x, ldx, nullptr, w_gate, w_up, ldw, false);
    if (workspace == nullptr) {
        *workspace_bytes = p.total;
        return ZOPT_OK;
    }
    if (w_gate == nullptr || w_up == nullptr || (T > 0 && (x == nullptr || h == nullptr))) return ZOPT_ERR_NULL;
    const bool keep = g8 != nullptr || g_scale != nullptr || u8 != nullptr || u_scale != nullptr;
    if (keep && T > 0 && (g8 == nullptr || g_scale == nullptr || u8 == nullptr || u_scale == nullptr))
        return ZOPT_ERR_NULL;
    if (act != kActSilu && act != kActGelu) return ZOPT_ERR_HYPER;
    const zopt_status st = workspace_check(p.total, workspace, *workspace_bytes);
    if (st != ZOPT_OK) return st;
    if (T == 0) return ZOPT_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    Preps preps;
    preps.place(p.x, ldx, ws);
    preps.place(p.wg, ldw, ws);
    preps.place(p.wu, ldw, ws);
    ZOPT_TRY(preps.run(s));
    Product both = p.products(kTgGlu);
    TgLaunch &L = both.L;
    L.act = act;
    L.h = h;
    L.ldc = ldh;
    L.g8 = g8;
    L.gs = g_scale;
    L.u8 = u8;
    L.us = u_scale;
    return device(both.run(false, false, ws + p.part, s));
}

ZOPT_EXPORT zopt_status zopt_glu_backward(int64_t T, int64_t D, int64_t F, const uint16_t *dh, int64_t lddh,
                                          const uint16_t *x, int64_t ldx, const uint8_t *x8, const uint8_t *x_scale,
                                          const uint16_t *w_gate, const uint16_t *w_up, int64_t ldw, int32_t act,
                                          const uint8_t *g8, const uint8_t *g_scale, const uint8_t *u8,
                                          const uint8_t *u_scale, uint16_t *h, int64_t ldh, uint16_t *dx,
                                          int64_t lddx, uint16_t *dw_gate, uint16_t *dw_up, int64_t lddw,
                                          void *workspace, size_t *workspace_bytes, void *stream) {
    if (workspace_bytes == nullptr) return ZOPT_ERR_NULL;
    if (!range(T, 0, kMaxRows) || !range(D, 1, kMaxSide) || !range(F, 1, kMaxSide)) return ZOPT_ERR_SIZE;
    if (!stride_ok(lddh, F) || !stride_ok(ldw, D) || (x8 == nullptr && !stride_ok(ldx, D))) return ZOPT_ERR_SIZE;
    if (!stride_ok(lddx, D) || !stride_ok(lddw, D) || (h != nullptr && !stride_ok(ldh, F))) return ZOPT_ERR_SIZE;
    GluPlan p = glu_plan(T, D, F, x, ldx, x8, w_gate, w_up, ldw, true);
    if (workspace == nullptr) {
        *workspace_bytes = p.total;
        return ZOPT_OK;
    }
    if (w_gate == nullptr || w_up == nullptr || dw_gate == nullptr || dw_up == nullptr) return ZOPT_ERR_NULL;
    if (T > 0 && (dh == nullptr || dx == nullptr)) return ZOPT_ERR_NULL;
    if (T > 0 && (x8 == nullptr ? x == nullptr : x_scale == nullptr)) return ZOPT_ERR_NULL;
    const bool kept = g8 != nullptr || g_scale != nullptr || u8 != nullptr || u_scale != nullptr;
    if (kept && T > 0 && (g8 == nullptr || g_scale == nullptr || u8 == nullptr || u_scale == nullptr))
        return ZOPT_ERR_NULL;
    if (act != kActSilu && act != kActGelu) return ZOPT_ERR_HYPER;
    const zopt_status st = workspace_check(p.total, workspace, *workspace_bytes);
    if (st != ZOPT_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    if (T == 0) {
        ZOPT_TRY(launch_fill_zero(dw_gate, lddw, F, D, s));
        ZOPT_TRY(launch_fill_zero(dw_up, lddw, F, D, s));
        return ZOPT_OK;
    }
    uint16_t *dg = reinterpret_cast<uint16_t *>(ws + p.dg), *du = reinterpret_cast<uint16_t *>(ws + p.du);
    Preps preps;
    if (x8 != nullptr)
        preps.unpack(p.x, x8, x_scale, ws);
    else
        preps.place(p.x, ldx, ws);
    preps.place(p.wg, ldw, ws);
    preps.place(p.wu, ldw, ws);
    if (kept) {
        TgPrep &j = preps.add(kPrepBack, T, F);
        j.q = g8;
        j.scale = g_scale;
        j.q2 = u8;
        j.scale2 = u_scale;
        j.src = dh;
        j.ld = lddh;
        j.act = act;
        j.dst = dg;
        j.dst2 = du;
        j.dst_ld = p.fp;
        j.h = h;
        j.h_ld = ldh;
    }
    ZOPT_TRY(preps.run(s));
    if (!kept) {
        Product both = p.products(kTgGluBack);
        TgLaunch &L = both.L;
        L.act = act;
        L.h = h;
        L.ldc = ldh;
        L.dh = dh;
        L.lddh = lddh;
        L.dg = dg;
        L.du = du;
        L.lddg = p.fp;
        ZOPT_TRY(both.run(false, false, ws + p.part, s));
    }
    Product gx = p.dx(ws);
    gx.L.prob[0].out = dx;
    gx.L.ldc = lddx;
    ZOPT_TRY(gx.run(false, true, ws + p.part, s));
    Product gw = p.dw(ws);
    gw.L.prob[0].out = dw_gate;
    gw.L.prob[1].out = dw_up;
    gw.L.ldc = lddw;
    return device(gw.run(true, true, ws + p.part, s));
}

ZOPT_EXPORT zopt_status zopt_act8_pack(int64_t rows, int64_t cols, const uint16_t *x, int64_t ldx, uint8_t *q,
                                       uint8_t *scale, void *stream) {
    if (!range(rows, 0, kMaxRows) || !range(cols, 1, kMaxSide) || !stride_ok(ldx, cols)) return ZOPT_ERR_SIZE;
    if (rows == 0) return ZOPT_OK;
    if (x == nullptr || q == nullptr || scale == nullptr) return ZOPT_ERR_NULL;
    return device(launch_act8_pack(x, ldx, rows, cols, q, scale, static_cast<hipStream_t>(stream)));
}

ZOPT_EXPORT zopt_status zopt_act8_unpack(int64_t rows, int64_t cols, const uint8_t *q, const uint8_t *scale,
                                         uint16_t *x, int64_t ldx, void *stream) {
    if (!range(rows, 0, kMaxRows) || !range(cols, 1, kMaxSide) || !stride_ok(ldx, cols)) return ZOPT_ERR_SIZE;
    if (rows == 0) return ZOPT_OK;
    if (x == nullptr || q == nullptr || scale == nullptr) return ZOPT_ERR_NULL;
    return device(launch_act8_unpack(q, scale, rows, cols, x, ldx, static_cast<hipStream_t>(stream)));
}

ZOPT_EXPORT zopt_status zopt_act8_wgrad(int64_t T, int64_t N, int64_t D, const uint16_t *dy, int64_t lddy,
                                        const uint8_t *q, const uint8_t *scale, uint16_t *dw, int64_t lddw,
                                        void *workspace, size_t *workspace_bytes, void *stream) {
    if (workspace_bytes == nullptr) return ZOPT_ERR_NULL;
    if (!range(T, 0, kMaxRows) || !range(N, 1, kMaxSide) || !range(D, 1, kMaxSide)) return ZOPT_ERR_SIZE;
    if (!stride_ok(lddy, N) || !stride_ok(lddw, D)) return ZOPT_ERR_SIZE;
    Carve c;
    Input x = input(nullptr, D, T, D, true, c);
    Input y = input(dy, lddy, T, N, false, c);
    Product g(kTgStore, N, D, segment(across(y, 0, T), across(x, 0, T)));
    const size_t part = c.take(T > 0 ? g.parts() : 0);
    if (workspace == nullptr) {
        *workspace_bytes = c.total();
        return ZOPT_OK;
    }
    if (dw == nullptr || (T > 0 && (dy == nullptr || q == nullptr || scale == nullptr))) return ZOPT_ERR_NULL;
    const zopt_status st = workspace_check(c.total(), workspace, *workspace_bytes);
    if (st != ZOPT_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    if (T == 0) return device(launch_fill_zero(dw, lddw, N, D, s));
    Preps preps;
    preps.unpack(x, q, scale, ws);
    preps.place(y, lddy, ws);
    ZOPT_TRY(preps.run(s));
    g.L.prob[0].seg[0] = segment(across(y, 0, T), across(x, 0, T));
    g.L.prob[0].out = dw;
    g.L.ldc = lddw;
    return device(g.run(true, true, ws + part, s));
}
