// train_gemm.hip -- the matrix products of the gradient operators on bf16
// matrix cores (gfx950), with their epilogues.
//
// C = sum over segments of A B^T; each operand is read as it lies in memory,
// along the reduction index (row-major) or across it (k-major, through
// transposing LDS reads), so no product needs a transposed copy:
//
//   logits, gate / up   x [T, D], w [V, D]      both row-major
//   dX                  P [T, V], w [V, D]      w k-major
//   dW                  P [T, V], x [T, D]      both k-major
//
// The MFMA takes B's fragment first, so a lane holds four consecutive columns
// of one row of C: lane (c, q) = (l % 16, l / 16) of 16 x 16 block (i, j) has
// row 16 i + c, columns 4 q .. 4 q + 3 of block j.  For a row-major B the rows
// are put into LDS in an order that makes the columns of blocks 2 j' and
// 2 j' + 1 together eight consecutive ones of a 32-column span (lane q:
// columns 8 q .. 8 q + 7), so that epilogues work on and store 16 bytes.
#include <utility>

#include "train_internal.h"

namespace zopt {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

#define LDS_ADDR(p) ((__attribute__((address_space(3))) void *)(p))

constexpr int kBK = 32;  // reduction elements per stage

// output tiles
enum Tile : int { kTile64 = 64, kTile128 = 128, kTile256x128 = 192, kTile256 = 256 };

// f(0), f(1), ... with the index as a type
template <int... M, class F>
__device__ __forceinline__ void for_each(std::integer_sequence<int, M...>, F f) {
    (f(std::integral_constant<int, M>{}), ...);
}

// The lane's index, computed afresh where it is used between tiles, so that
// what is derived from it holds no registers across the main loop.
__device__ __forceinline__ int lane_id() {
    int l;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
    return l;
}

// Tile t of a tiles_m x tiles_n grid: bands of 16 tile rows, in a band groups
// of 8 columns, in a group runs of 4 rows, column by column.  A round of 256
// tiles is then about 16 x 16 and an XCD's 32 about 4 x 8: few operand panels
// in each L2, and few of them read more than once from HBM.
__device__ __forceinline__ void tile_at(int t, int tm, int tn, int &ti, int &tj) {
    const int band = t / (16 * tn), r0 = band * 16;
    t -= band * 16 * tn;
    const int h = tm - r0 < 16 ? tm - r0 : 16;
    const int group = t / (8 * h), c0 = group * 8;
    t -= group * 8 * h;
    const int w = tn - c0 < 8 ? tn - c0 : 8;
    const int run = t / (4 * w), q0 = run * 4;
    t -= run * 4 * w;
    const int hh = h - q0 < 4 ? h - q0 : 4;
    tj = c0 + t / hh;
    ti = r0 + q0 + t % hh;
}

// v of the lanes (c, q), (c, q ^ 1) and (c, q), (c, q ^ 2): the two values, in
// one order on both sides, by gfx950's row and half exchanges
struct Pair {
    uint32_t a, b;
};
__device__ __forceinline__ Pair across16(uint32_t v) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return {r[0], r[1]};
}
__device__ __forceinline__ Pair across32(uint32_t v) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return {r[0], r[1]};
}
// maximum / sum over the four lanes of a row (q = 0 .. 3)
__device__ __forceinline__ float quad_max(float v) {
    Pair p = across16(__float_as_uint(v));
    v = fmaxf(__uint_as_float(p.a), __uint_as_float(p.b));
    p = across32(__float_as_uint(v));
    return fmaxf(__uint_as_float(p.a), __uint_as_float(p.b));
}
__device__ __forceinline__ float quad_sum(float v) {
    Pair p = across16(__float_as_uint(v));
    v = __uint_as_float(p.a) + __uint_as_float(p.b);
    p = across32(__float_as_uint(v));
    return __uint_as_float(p.a) + __uint_as_float(p.b);
}
__device__ __forceinline__ uint32_t quad_umax(uint32_t v) {
    Pair p = across16(v);
    v = p.a > p.b ? p.a : p.b;
    p = across32(v);
    return p.a > p.b ? p.a : p.b;
}

// Row statistics and exponentials of a logits tile.  A wave's 64 columns are
// one statistics group: m = their largest logit, s = the sum of exp(z - m),
// and e = exp(z - m) in (0, 1] kept in fp16 (11 bits; what is lost below
// 2^-14 is under 2^-25 of the group's largest).  exp(z - m) is taken as
// 2^((z - m) log2 e), the difference first: m's own exponential is then exactly
// 1, so that s >= 1 and no row's loss is negative, and the error does not grow
// with |m| (a multiply-add z log2 e - m log2 e, one operation less, is off by
// 2^-24 of |m| log2 e: losses of sure rows down to -8e-5 at |m| = 2048).
// Bound by the vector units and the stores: on [8192, 768] x [768, 50304] the
// products alone take 0.46 ms, the statistics 0.09 more (half of it the
// exponentials, at a quarter of the rate), the 824 MB of e 0.12.
// target: those of the lane's rows, or -1 (a column that does not exist).
template <int FM>
__device__ __forceinline__ void xent_epilogue(const TgLaunch &L, tg_f32x4 (&acc)[FM][4], int R0, int C0,
                                              const int (&target)[FM]) {
    const int lane = lane_id(), c = lane & 15, q = lane >> 4;
    if (C0 >= L.N) return;  // (lde - N < 64: no column of e lies in a group past N's last)
    float2 *stats = L.stats + (int64_t)(R0 + c) * L.ldstat + C0 / kXentGroup;
    uint16_t *e = L.e + (int64_t)(R0 + c) * L.lde + C0 + q * 8;
    const int rows = L.M - R0 - c, cols = L.N - C0 - q * 8;
    const bool whole = C0 + 64 <= L.N, keep = L.e != nullptr;
    constexpr float kLog2e = 1.4426950408889634f;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        float z[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) z[k] = acc[i][k >> 2][k & 3];
        if (!whole) {
#pragma unroll
            for (int k = 0; k < 16; ++k) z[k] = (k >> 3) * 32 + (k & 7) < cols ? z[k] : -INFINITY;
        }
        float m = z[0];
#pragma unroll
        for (int k = 1; k < 16; ++k) m = fmaxf(m, z[k]);
        m = quad_max(m);
        const bool live = i * 16 < rows;
        // the target's logit, where it is one of this lane's columns
        const int rel = target[i] - C0 - q * 8;
        if (live && (rel & ~39) == 0) {
            const int at = (rel >> 5) * 8 + (rel & 7);
            float v = z[0];
#pragma unroll
            for (int k = 1; k < 16; ++k) v = at == k ? z[k] : v;
            L.zt[R0 + c + i * 16] = v;
        }
        // a group of -inf alone: exponentials 0, not NaN
        const float ref = m == -INFINITY ? 0.0f : m;
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            z[k] = __builtin_amdgcn_exp2f((z[k] - ref) * kLog2e);
            s += z[k];
        }
        s = quad_sum(s);
        if (live) {
            if (q == 0) *stats = make_float2(m, s);
            if (keep) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const tg_u32x4 p{tg_pack_f16(z[8 * h], z[8 * h + 1]), tg_pack_f16(z[8 * h + 2], z[8 * h + 3]),
                                     tg_pack_f16(z[8 * h + 4], z[8 * h + 5]), tg_pack_f16(z[8 * h + 6], z[8 * h + 7])};
                    // (the markers keep the two from being merged into one
                    // ordinary store)
                    if (L.past) {
                        asm volatile("; past the caches");
                        tg_store<true>(e + h * 32, p);
                        asm volatile("; past the caches");
                    } else {
                        tg_store<false>(e + h * 32, p);
                    }
                }
            }
        }
        stats += 16 * L.ldstat;
        e += 16 * L.lde;
        __builtin_amdgcn_sched_barrier(0);
    }
}

__device__ __forceinline__ tg_u32x4 pack8(const float (&v)[8]) {
    return tg_u32x4{tg_pack_bf16(v[0], v[1]), tg_pack_bf16(v[2], v[3]), tg_pack_bf16(v[4], v[5]),
                    tg_pack_bf16(v[6], v[7])};
}
__device__ __forceinline__ void unpack8(tg_u32x4 p, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(p[k] << 16);
        v[2 * k + 1] = __uint_as_float(p[k] & 0xFFFF0000u);
    }
}

// One row's 32-column block of an 8-bit checkpoint, eight values in each of
// the lanes q = 0 .. 3 of column c: the scale from the largest magnitude of
// all four, then the lane's eight bytes.
__device__ __forceinline__ void act8_store(const float (&v)[8], int n, uint8_t *qrow, uint8_t *srow, int col,
                                           int q, bool live) {
    uint32_t big = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t b = __float_as_uint(v[k]) & 0x7FFFFFFFu;
        big = k < n && b > big ? b : big;
    }
    const uint32_t byte = tg_scale_byte(quad_umax(big));
    if (!live) return;
    if (n > 0) tg_store8b(qrow + col, tg_pack_e4m3(v, byte), n);
    if (q == 0) srow[col >> 5] = (uint8_t)byte;
}

// Gate and up columns of a tile: blocks 0, 1 are the gate's 32 columns, 2, 3
// the up projection's same columns; C0 is the first of them.
template <int FM, bool BACK>
__device__ __forceinline__ void glu_epilogue(const TgLaunch &L, tg_f32x4 (&acc)[FM][4], int R0, int C0) {
    const int lane = lane_id(), c = lane & 15, q = lane >> 4;
    const int F = L.N;
    if (C0 >= F) return;
    const int col = C0 + q * 8;
    const int n = F - col > 8 ? 8 : F - col < 0 ? 0 : F - col;
    const int64_t blocks = (F + 31) / 32;
    // (dh is read three row blocks ahead of the stores: loads and stores are
    // counted in order, so a load behind a store waits for it)
    constexpr int kAhead = FM < 3 ? FM : 3;
    tg_u32x4 ahead[kAhead];
    auto fetch = [&](int i) __attribute__((always_inline)) {
        const int row = R0 + i * 16 + c;
        if (i < FM && row < L.M && n > 0) ahead[i % kAhead] = tg_load8h(L.dh + (int64_t)row * L.lddh + col, n);
    };
    if constexpr (BACK) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(i);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int row = R0 + i * 16 + c;
        const bool live = row < L.M;
        float g[8], u[8], h[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            g[k] = acc[i][k >> 2][k & 3];
            u[k] = acc[i][2 + (k >> 2)][k & 3];
        }
        if constexpr (!BACK) {
#pragma unroll
            for (int k = 0; k < 8; ++k) h[k] = tg_act(g[k], L.act).a * u[k];
            if (live && n > 0) tg_store8h(L.h + (int64_t)row * L.ldc + col, pack8(h), n);
            if (L.g8 != nullptr) {
                act8_store(g, n, L.g8 + (int64_t)row * F, L.gs + (int64_t)row * blocks, col, q, live);
                act8_store(u, n, L.u8 + (int64_t)row * F, L.us + (int64_t)row * blocks, col, q, live);
            }
        } else {
            if (live && n > 0) {
                float dh[8], dg[8], du[8];
                unpack8(ahead[i % kAhead], dh);
                fetch(i + kAhead);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const TgActValue a = tg_act(g[k], L.act);
                    h[k] = a.a * u[k];
                    du[k] = k < n ? dh[k] * a.a : 0.0f;
                    dg[k] = k < n ? dh[k] * u[k] * a.da : 0.0f;
                }
                // (the padded row has room for all eight)
                *reinterpret_cast<tg_u32x4 *>(L.dg + (int64_t)row * L.lddg + col) = pack8(dg);
                *reinterpret_cast<tg_u32x4 *>(L.du + (int64_t)row * L.lddg + col) = pack8(du);
                if (L.h != nullptr) tg_store8h(L.h + (int64_t)row * L.ldc + col, pack8(h), n);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// A tile of sums: alpha * acc to bf16; SUM: plus earlier fp32 sums, or kept as
// such for a later call.
// PERM: the column order of a row-major B (eight consecutive per lane).
template <int FM, int FN, bool PERM, bool SUM>
__device__ __forceinline__ void store_epilogue(const TgLaunch &L, const TgProblem &P, float alpha,
                                               tg_f32x4 (&acc)[FM][FN], int R0, int C0) {
    const int lane = lane_id(), c = lane & 15, q = lane >> 4;
    // the lane's first column, and the one of block j
    const int first = C0 + (PERM ? q * 8 : q * 4);
    auto at = [](int j) __attribute__((always_inline)) { return PERM ? (j >> 1) * 32 + (j & 1) * 4 : j * 16; };
    const int rows = L.M - R0 - c, cols = L.N - first;  // what is left from the lane's first place on
    const bool in = SUM && L.sum_in != 0;
    float *s = P.sum + (int64_t)(R0 + c) * L.ldsum + first;  // (rows of fp32 sums are padded to a multiple of 4)
    const int64_t sstep = 16 * L.ldsum;
    uint16_t *o = P.out + (int64_t)(R0 + c) * L.ldc + first;
    const int64_t step = 16 * L.ldc;
    // the earlier sums are read a row block ahead of the stores: loads and
    // stores are counted in order, so a load behind a store waits for it
    tg_f32x4 ahead[FN];
    auto fetch = [&](int i) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
            if (i < FM && i * 16 < rows && at(j) < cols)
                ahead[j] = *reinterpret_cast<const tg_f32x4 *>(s + i * sstep + at(j));
    };
    if (in) fetch(0);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        tg_f32x4 v[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) v[j] = acc[i][j];
        if (in) {
#pragma unroll
            for (int j = 0; j < FN; ++j) v[j] += ahead[j];
            fetch(i + 1);
        }
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            if (i * 16 < rows && at(j) < cols) {
                if (SUM && L.sum_out) {
                    *reinterpret_cast<tg_f32x4 *>(s + i * sstep + at(j)) = v[j];
                } else {
                    const tg_f32x4 x = v[j] * alpha;
                    const tg_u32x2 p{tg_pack_bf16(x[0], x[1]), tg_pack_bf16(x[2], x[3])};
                    if (at(j) + 4 <= cols) {
                        tg_store(o + at(j), p);
                    } else {
                        o[at(j)] = (uint16_t)p.x;
                        if (at(j) + 1 < cols) o[at(j) + 1] = (uint16_t)(p.x >> 16);
                        if (at(j) + 2 < cols) o[at(j) + 2] = (uint16_t)p.y;
                    }
                }
            }
        }
        o += step;
        __builtin_amdgcn_sched_barrier(0);
    }
}

// The factor of the outputs, in a scalar register: read once, before the main
// loop (a load among the stores would wait for the operands in flight).
__device__ __forceinline__ float read_alpha(const TgLaunch &L) {
    float a = 1.0f;
    if (L.alpha != nullptr) a = *L.alpha;
    return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(a)));
}

// What becomes of a wave's sums, BM / WR rows from R0 and 64 columns (32 of
// the gate and of the up projection) from C0 on.
template <int EPI, bool BKM, int FM>
__device__ __forceinline__ void finish(const TgLaunch &L, int prob, float alpha, tg_f32x4 (&acc)[FM][4], int R0,
                                       int C0, const int (&target)[FM]) {
    if constexpr (EPI == kTgXent)
        xent_epilogue<FM>(L, acc, R0, C0, target);
    else if constexpr (EPI == kTgGlu || EPI == kTgGluBack)
        glu_epilogue<FM, EPI == kTgGluBack>(L, acc, R0, C0);
    else
        store_epilogue<FM, 4, !BKM, EPI == kTgSum>(L, L.prob[prob], alpha, acc, R0, C0);
}

// Tiles.  A BM x BN tile per workgroup, its WR x WC waves BM / WR x 64 each,
// from 16 x 16 x 32 MFMAs with fp32 accumulators; STAGES LDS buffers; WPE
// waves per SIMD.
template <int TILE>
struct Cfg;
template <>
struct Cfg<kTile256> { static constexpr int BM = 256, BN = 256, WR = 2, WC = 4, STAGES = 4, WPE = 2; };
template <>
struct Cfg<kTile256x128> { static constexpr int BM = 256, BN = 128, WR = 2, WC = 2, STAGES = 3, WPE = 2; };
template <>
struct Cfg<kTile128> { static constexpr int BM = 128, BN = 128, WR = 2, WC = 2, STAGES = 4, WPE = 2; };
template <>
struct Cfg<kTile64> { static constexpr int BM = 64, BN = 64, WR = 4, WC = 1, STAGES = 4, WPE = 4; };

// s_waitcnt: vmcnt <= n and lgkmcnt = 0 (gfx9 field layout: vmcnt[3:0],
// expcnt[6:4], lgkmcnt[11:8], vmcnt high bits[15:14])
#define WAIT_VM_LGKM0(n) ((((n) & 15) | (((n) >> 4) << 14) | (7 << 4)))

// A wave's sums of part `split` of split tile t, in register order (16 bytes a
// lane).
template <int FM, int NW>
__device__ __forceinline__ void keep_part(const TgLaunch &L, int t, int split, int wave, tg_f32x4 (&acc)[FM][4]) {
    tg_f32x4 *p = reinterpret_cast<tg_f32x4 *>(L.part) +
                  (((int64_t)t * L.splits + split) * NW + wave) * (FM * 4 * 64) + lane_id();
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j * 64] = acc[i][j];
        p += 4 * 64;
        __builtin_amdgcn_sched_barrier(0);
    }
}

// The main loop.  The reduction advances in stages of 32 through STAGES LDS
// buffers that buffer_load ... lds fills ahead (16 bytes a lane;
// a lane outside the operand reads past its descriptor's end, which gives
// zeros).  A stage's body: barrier (everyone's loads of the next stage have
// landed and everyone has read this one's fragments) -> loads of the stage
// STAGES ahead into the buffer just freed -> the next stage's fragments, read
// between this stage's MFMAs -> wait for those reads and for this wave's
// loads of the stage after.
//
// A row-major operand's rows then come in pieces of 64 bytes, half a cache
// line, and every line is asked for twice.  So with four buffers and A
// row-major they hold two PAIRS of stages: all loads of a pair, 128 bytes a
// row, go out in the body of an odd stage, past its barrier, and are waited for
// at the end of the next body, which needs no barrier.  Measured: the products
// of two row-major operands 5 to 8% faster ([8192, 4096] x [4096, 28672] 1.42 ms
// for 1.52), with B k-major 1 to 2% on 256 x 256 tiles, 7% slower on the smaller
// ones; with both k-major 3% slower (nothing to gain, and the loads are one
// stage closer to their use), so neither takes it.
//
// The kernel is persistent: one round of resident workgroups walks all tiles,
// and from a tile's last STAGES stages on the loads are those of the
// workgroup's next tile, so that its operands arrive while this one is
// finished and stored.  Segments and parts are of whole pairs of stages, tiles
// padded with zero stages to four at least.
//
// LDS layouts: row-major rows of 64 bytes, 16-byte chunk c of row r at slot
// c ^ ((r >> 1) & 3), in pairs 128 bytes and c ^ (r & 7); k-major rows of 2 BM (2 BN) bytes, 32-byte unit u of row r at
// unit u ^ qsw(r), read with ds_read_b64_tr_b16: lane 4 q + p of a 16-lane
// group addresses row +q, columns 4 p .. 4 p + 3 of a 4 x 16 block, and lane
// i receives rows +0 .. +3 of column i.  Both spread each read over all
// banks.  The reads are inline assembly: as ordinary loads the compiler cannot
// tell them from the copies in flight into other buffers and may wait for
// those.  Each is waited for within the stage's body.
//
// Bound by the matrix cores and by a stage's synchronisation: measured on the
// 8192-token products of a 4096 x 14336 block, 256 x 256 tiles run at 1.29
// PFLOP/s with both operands k-major (1.50 ms), 1.37 with B alone (1.41 ms), 1.32
// with the gate's epilogue and checkpoints (1.45 ms); by counters the matrix cores
// are 63%, 67% and 64% busy at 2.0 to 2.1 GHz, LDS 24 to 25%, no bank conflicts.
// A library product of the same sizes reaches 1.20, 1.41 and (alone, without an
// epilogue) 1.57.  Measured without
// gain: fragment reads late, early or opposite in the two waves of a SIMD (all
// within 1%), XCDs started at different times, two 256 x 128 workgroups a CU
// for large products (1.5 times the operand traffic: 9.0 ms for 7.0 on
// [8192, 4096] x [4096, 131072]; used where tiles are few).
template <int TILE, int EPI, bool AKM, bool BKM>
__global__ __launch_bounds__(Cfg<TILE>::WR *Cfg<TILE>::WC * 64)
__attribute__((amdgpu_waves_per_eu(Cfg<TILE>::WPE))) void tg_kernel(TgLaunch L) {
    using C = Cfg<TILE>;
    constexpr int BM = C::BM, BN = C::BN, WR = C::WR, WC = C::WC, NW = WR * WC, kStages = C::STAGES;
    constexpr int WTM = BM / WR, FM = WTM / 16, FN = 4;
    static_assert(BN / WC == 64, "a wave holds 64 columns");
    constexpr int OPA = BM * kBK * 2, OPB = BN * kBK * 2, STAGE = OPA + OPB;
    constexpr bool PAIRS = !AKM && kStages == 4 && (!BKM || TILE == kTile256);  // (see above)
    constexpr int SPL = PAIRS ? 2 : 1, ROW = 64 * SPL;  // stages a load; bytes of a row-major row
    constexpr int LA = SPL * OPA / 1024 / NW, LB = SPL * OPB / 1024 / NW, LPS = LA + LB;  // of a wave, each SPL stages
    static_assert(LA * NW * 1024 == SPL * OPA && LB * NW * 1024 == SPL * OPB, "whole kilobytes");
    constexpr int QRA = 2 * BM, QRB = 2 * BN;  // k-major row bytes
    constexpr bool GLU = EPI == kTgGlu || EPI == kTgGluBack;
    static_assert(!GLU || NW % 4 == 0, "a wave loads rows of the gate or of the up projection");
    constexpr int BO = GLU ? BN / 2 : BN;  // output columns of a tile
    constexpr int kOut = 0x7FFFFFF0;       // a byte offset past every descriptor
    // exponentials: the targets of a tile's rows, of this tile and the next
    constexpr bool XENT = EPI == kTgXent;
    constexpr int TGB = XENT ? (BM * 8 < 1024 ? 1024 : BM * 8) : 0;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kStages * STAGE + 2 * TGB];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave / WC, wc = wave % WC;
    constexpr bool PLAIN = EPI == kTgStore || EPI == kTgSum;
    const int grid = gridDim.x - (PLAIN && L.sum_up.loss != nullptr ? 1 : 0);
    if constexpr (PLAIN) {
        if ((int)blockIdx.x == grid) {
            tg_total<NW * 64>(L.sum_up);
            return;
        }
    }
    const uint32_t lds_base =
        (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t *)lds);

    auto qsw = [](int r, int width) __attribute__((always_inline)) {
        return width >= 128 ? (r & 3) | (((r >> 3) & 1) << 2) : ((r >> 1) & 1) | (((r >> 3) & 1) << 1);
    };

    struct Tile {
        int t, prob, split, m0, n0, stage0, live, stages;  // split: -1 whole; live: real stages; stages: padded
    };
    // slot -> tile (false: a padding slot).  Workgroups go to the 8 XCDs in
    // turn; XCD x takes the x-th contiguous eighth of each round of resident
    // tiles, and consecutive tiles form blocks of the grid, so that each L2
    // serves few operand panels.
    auto locate = [&](int slot, Tile &T) __attribute__((always_inline)) -> bool {
        const int base = slot - slot % grid;
        const int rem = L.padded - base < grid ? L.padded - base : grid;
        int t = base + (slot & 7) * (rem >> 3) + ((slot - base) >> 3);
        if (t >= L.total) return false;
        // (parts of the tiles that are split: all first ones, all second ones, ...)
        T.split = -1;
        if (t >= L.whole && L.splits > 1) {
            const int rest = L.tiles - L.whole;
            T.split = (t - L.whole) / rest;
            t -= T.split * rest;
        }
        T.t = t;
        const int per = L.tiles_m * L.tiles_n;
        T.prob = t >= per ? 1 : 0;
        int ti, tj;
        tile_at(t - T.prob * per, L.tiles_m, L.tiles_n, ti, tj);
        T.m0 = ti * BM;
        T.n0 = tj * BO;
        const TgProblem &P = L.prob[T.prob];
        const int all = P.seg[0].stages + (PLAIN && P.nseg > 1 ? P.seg[1].stages : 0);
        T.stage0 = T.split < 0 ? 0 : T.split * L.split_stages;
        T.live = all - T.stage0;
        if (T.split >= 0 && T.live > L.split_stages) T.live = L.split_stages;
        T.stages = T.live < 4 ? 4 : T.live;  // (the switch to the next tile is kStages before)
        return true;
    };
    auto seek = [&](int slot, Tile &T) __attribute__((always_inline)) -> int {
        for (; slot < L.padded; slot += grid)
            if (locate(slot, T)) return slot;
        return -1;
    };

    // ------------------------------------------------ the load stream
    // Of each operand: the tile's corner at the stream's current reduction
    // index, what is left of the reduction, the byte extent of the panel's
    // rows before the last (row-major) or of one row (k-major), and each
    // lane's byte offset per kilobyte.
    const uint16_t *pa = nullptr, *pb = nullptr;
    int ka = 0, kb = 0, lda = 0, ldb = 0, ea = 0, eb = 0, seg_left = 0, total_left = 0;
    int sprob = 0, sm0 = 0, sn0 = 0;
    int va[PAIRS ? 1 : LA], vb[PAIRS ? 1 : LB];
    // row-major: the lane's row of a kilobyte's and its k offset
    const int krow = PAIRS ? lane >> 3 : lane >> 2;
    const int chunk8 = (PAIRS ? (lane & 7) ^ (lane >> 3) : (lane & 3) ^ ((lane >> 3) & 3)) << 3;
    // The wave's x-th kilobyte of an operand is number first + kx(x), such that
    // its offset differs from that of the first by whole rows.  (k-major, 512-byte
    // rows: kilobytes of the same swizzle; row-major pairs: a wave's LDS blocks
    // of B are 0, 1 of each four or 2, 3.)  With pairs a lane keeps the first's
    // offset, for registers, and adds the rows (kOut stays past every
    // descriptor: less than 2^32 in all); else it keeps all, 1% faster.
    constexpr bool spread_a = AKM ? BM == 256 : PAIRS, spread_b = BKM ? BN == 256 : PAIRS;
    static_assert((!spread_a || LA % 2 == 0) && (!spread_b || LB % 2 == 0), "kx runs over all kilobytes");
    auto kx = [](bool spread, int x) constexpr { return spread ? (x >> 1) * 2 * NW + (x & 1) * 2 : x * NW; };
    const int first_a = spread_a ? (wave >> 1) * 4 + (wave & 1) : wave;
    const int first_b = spread_b ? (wave >> 1) * 4 + (wave & 1) : wave;
    auto rows_a = [&](int x) __attribute__((always_inline)) -> int {
        return kx(spread_a, x) * (AKM ? 512 / BM : 16 / SPL);
    };
    auto rows_b = [&](int x) __attribute__((always_inline)) -> int {
        if (BKM) return kx(spread_b, x) * (512 / BN);
        return PAIRS ? (x >> 1) * (GLU ? NW / 4 : NW / 2) * 32 + (x & 1) * 4 : x * (GLU ? NW / 4 : NW / 2) * 32;
    };
    auto plus = [](int offset, int elements) __attribute__((always_inline)) -> int {
        return (int)((uint32_t)offset + (uint32_t)elements * 2u);
    };
    auto corner = [&](const TgOperand &o, bool km, int c0, int extent, int k0, const uint16_t *&p, int &k, int &ld,
                      int &e) __attribute__((always_inline)) {
        ld = (int)o.ld;
        k = o.k - k0;
        if (km) {
            p = o.p + (int64_t)k0 * o.ld + c0;
            e = (o.outer - c0) * 2;
        } else {
            p = o.p + (int64_t)c0 * o.ld + k0;
            const int left = o.outer - c0;
            e = ((left < extent ? left : extent) - 1) * ld * 2;
        }
    };
    auto open_segment = [&](int s, int k0) __attribute__((always_inline)) {
        const TgProblem &P = L.prob[sprob];
        const TgSegment &S = P.seg[s];
        seg_left = S.stages - k0 / kBK;
        corner(S.a, AKM, sm0, BM, k0, pa, ka, lda, ea);
        // gate / up: LDS blocks 0, 1 of each four hold the gate's rows (wave
        // w fills blocks w, w + NW, ...)
        corner(GLU && (wave & 2) ? P.seg[1].b : S.b, BKM, sn0, BO, k0, pb, kb, ldb, eb);
    };
    auto stream = [&](const Tile &T, bool live) __attribute__((always_inline)) {
        total_left = live ? T.live : 0;
        sprob = T.prob;
        sm0 = T.m0;
        sn0 = T.n0;
        const int s0 = L.prob[T.prob].seg[0].stages;
        if (PLAIN && T.stage0 >= s0)
            open_segment(1, (T.stage0 - s0) * kBK);
        else
            open_segment(0, T.stage0 * kBK);
        // k-major: kilobyte `kilo` holds 1024 / (2 width) k rows
        auto across = [&](int kilo, int width, int ld, int e) __attribute__((always_inline)) -> int {
            const int per = width / 8, r = kilo * (512 / width) + lane / per, s16 = lane % per;
            const int col = (((s16 >> 1) ^ qsw(r, width)) << 4) + ((s16 & 1) << 3);
            return col * 2 < e ? (r * ld + col) * 2 : kOut;
        };
        const int base_a = AKM ? across(first_a, BM, lda, ea) : ((first_a * (16 / SPL) + krow) * lda + chunk8) * 2;
        // row-major: LDS row n of 16-row block `blk` holds the tile's column
        // 32 (blk / 2) + 8 (n / 4) + 4 (blk % 2) + n % 4; gate / up: of the 32
        // columns of wave blk / 4
        const int blk = first_b / SPL, n = (first_b & (SPL - 1)) * 8 + krow;
        const int row = (GLU ? blk >> 2 : blk >> 1) * 32 + 8 * (n >> 2) + 4 * (blk & 1) + (n & 3);
        const int base_b = BKM ? across(first_b, BN, ldb, eb) : (row * ldb + chunk8) * 2;
#pragma unroll
        for (int x = 0; x < (PAIRS ? 1 : LA); ++x) va[x] = plus(base_a, rows_a(x) * lda);
#pragma unroll
        for (int x = 0; x < (PAIRS ? 1 : LB); ++x) vb[x] = plus(base_b, rows_b(x) * ldb);
    };
    auto extent = [&](bool km, int k, int ld, int e) __attribute__((always_inline)) -> int {
        if (total_left <= 0 || k <= 0) return 0;
        if (km) return ((k < kBK * SPL ? k : kBK * SPL) - 1) * ld * 2 + e;
        return e + k * 2;
    };
    // load y: A's kilobytes, then B's
    __amdgpu_buffer_rsrc_t ra, rb;
    auto open_stage = [&]() __attribute__((always_inline)) {
        ra = __builtin_amdgcn_make_buffer_rsrc((void *)pa, (short)0, extent(AKM, ka, lda, ea), 0x00020000);
        rb = __builtin_amdgcn_make_buffer_rsrc((void *)pb, (short)0, extent(BKM, kb, ldb, eb), 0x00020000);
    };
    auto gload = [&](int sbase, int y) __attribute__((always_inline)) {
        // (a chunk past the row's end would be the next row's)
        if (y < LA) {
            const int kilo = first_a + kx(spread_a, y);
            const int first = AKM || chunk8 < ka ? va[PAIRS ? 0 : y] : kOut;
            const int o = PAIRS ? plus(first, rows_a(y) * lda) : first;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, LDS_ADDR(&lds[sbase + kilo * 1024]), 16, o, 0, 0, 0);
        } else {
            const int x = y - LA, kilo = first_b + kx(spread_b, x);
            const int first = BKM || chunk8 < kb ? vb[PAIRS ? 0 : x] : kOut;
            const int o = PAIRS ? plus(first, rows_b(x) * ldb) : first;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, LDS_ADDR(&lds[sbase + SPL * OPA + kilo * 1024]), 16, o, 0, 0, 0);
        }
    };
    auto close_stage = [&]() __attribute__((always_inline)) {
        pa += AKM ? (int64_t)kBK * SPL * lda : kBK * SPL;
        pb += BKM ? (int64_t)kBK * SPL * ldb : kBK * SPL;
        ka -= kBK * SPL;
        kb -= kBK * SPL;
        total_left -= SPL;
        // (real stages left after a segment's last: there is a second one)
        if (PLAIN && (seg_left -= SPL) == 0 && total_left > 0) open_segment(1, 0);
    };

    // -------------------------------------------------- fragments and products
    const int fr = lane & 15, fh = lane >> 4;
    const int foff = fr * ROW + ((fh ^ (PAIRS ? fr & 7 : (fr >> 1) & 3)) << 4);
    const int tr = 8 * fh + ((lane >> 2) & 3), tp = lane & 3;
    const uint32_t tlane = lds_base + ((tp >> 1) << 4) + ((tp & 1) << 3);
    const uint32_t toffa = tlane + tr * QRA + ((qsw(tr, BM) ^ (wr * FM)) << 5);
    const uint32_t toffb = tlane + tr * QRB + ((qsw(tr, BN) ^ (wc * FN)) << 5);
    bf16x8 fa[2][FM], fb[2][FN];
    // block `blk` of an operand: unit (first + blk) ^ qsw(row), i.e. the
    // address of block 0 with blk's bits flipped
    auto tread = [&](uint32_t at, auto BLK, auto ROWB) __attribute__((always_inline)) {
        tg_u32x2 lo, hi;
        uint32_t t;
        asm volatile(
            "v_xor_b32 %2, %3, %4\n\tds_read_b64_tr_b16 %0, %2\n\tds_read_b64_tr_b16 %1, %2 offset:%5"
            : "=&v"(lo), "=&v"(hi), "=&v"(t)
            : "i"(decltype(BLK)::value << 5), "v"(at), "i"(4 * decltype(ROWB)::value));
        return __builtin_bit_cast(bf16x8, tg_u32x4{lo.x, lo.y, hi.x, hi.y});
    };
    auto rread = [&](uint32_t at, auto BLK) __attribute__((always_inline)) {
        tg_u32x4 v;
        asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(v) : "v"(at), "i"(decltype(BLK)::value * 16 * ROW));
        return __builtin_bit_cast(bf16x8, v);
    };
    const uint32_t roffa = lds_base + wr * WTM * ROW + foff, roffb = lds_base + SPL * OPA + wc * 64 * ROW + foff;
    // fragment y of a stage: A's blocks, then B's
    auto read = [&](int buf, int sbase, auto Y) __attribute__((always_inline)) {
        constexpr int y = decltype(Y)::value;
        if constexpr (y < FM) {
            if constexpr (AKM)
                fa[buf][y] = tread(toffa + sbase + (PAIRS ? buf * OPA : 0), Y, std::integral_constant<int, QRA>{});
            else
                fa[buf][y] = rread((PAIRS ? roffa ^ (buf << 6) : roffa) + sbase, Y);
        } else {
            constexpr int j = y - FM;
            if constexpr (BKM)
                fb[buf][j] = tread(toffb + sbase + SPL * OPA + (PAIRS ? buf * OPB : 0), std::integral_constant<int, j>{},
                                   std::integral_constant<int, QRB>{});
            else
                fb[buf][j] = rread((PAIRS ? roffb ^ (buf << 6) : roffb) + sbase, std::integral_constant<int, j>{});
        }
    };
    // (after a wait: nothing that uses the fragments moves above it)
    auto tie = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FM; ++i) asm volatile("" : "+v"(fa[buf][i]));
#pragma unroll
        for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(fb[buf][j]));
    };
    tg_f32x4 acc[FM][FN];
    // steps of a stage's body: product m, then one load or fragment read
    auto steps = [&](auto PAR, int cbase, int nbase) __attribute__((always_inline)) {
        constexpr int par = decltype(PAR)::value, loads = PAIRS && par == 0 ? 0 : LPS;
        constexpr int kSteps = FM * FN > loads + FM + FN ? FM * FN : loads + FM + FN;
        for_each(std::make_integer_sequence<int, kSteps>{}, [&](auto MM) __attribute__((always_inline)) {
            constexpr int m = decltype(MM)::value;
            if constexpr (m < FM * FN) {
                constexpr int i = m / FN, j = m % FN;
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[par][j], fa[par][i], acc[i][j], 0, 0, 0);
            }
            if constexpr (m < loads)
                gload(cbase, m);
            else if constexpr (m - loads < FM + FN)
                read(par ^ 1, nbase, std::integral_constant<int, m - loads>{});
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    int cur = 0;
    auto body = [&](auto PAR) __attribute__((always_inline)) {
        constexpr int par = decltype(PAR)::value;
        if constexpr (PAIRS) {
            const int other = cur ^ (2 * STAGE);
            if constexpr (par == 0) {
                steps(PAR, 0, cur);
                __builtin_amdgcn_s_waitcnt(WAIT_VM_LGKM0(0));
            } else {
                __builtin_amdgcn_s_barrier();
                open_stage();
                __builtin_amdgcn_sched_barrier(0);
                steps(PAR, cur, other);
                close_stage();
                __builtin_amdgcn_s_waitcnt(WAIT_VM_LGKM0(63));
                cur = other;
            }
            __builtin_amdgcn_sched_barrier(0);
            tie(par ^ 1);
            return;
        }
        const int nxt = cur + 1 == kStages ? 0 : cur + 1;
        __builtin_amdgcn_s_barrier();
        open_stage();
        __builtin_amdgcn_sched_barrier(0);
        steps(PAR, cur * STAGE, nxt * STAGE);
        close_stage();
        __builtin_amdgcn_s_waitcnt(WAIT_VM_LGKM0((kStages - 2) * LPS));
        __builtin_amdgcn_sched_barrier(0);
        tie(par ^ 1);
        cur = nxt;
    };

    // the targets of a tile's rows, 128 a wave instruction, straight to LDS
    auto load_targets = [&](const Tile &T, int which) __attribute__((always_inline)) {
        if constexpr (XENT) {
            if (wave * 128 < BM) {
                const int left = (L.M - T.m0 < BM ? L.M - T.m0 : BM) * 8;
                const __amdgpu_buffer_rsrc_t rt = __builtin_amdgcn_make_buffer_rsrc(
                    (void *)(L.target + T.m0), (short)0, left, 0x00020000);
                const int off = (wave * 64 + lane_id()) * 16;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rt, LDS_ADDR(&lds[kStages * STAGE + which * TGB + wave * 1024]), 16, off, 0, 0, 0);
            }
        }
    };
    int which = 0;
    // ... and read back, those of the lane's rows; outside 0 .. 2^31 - 1: -1
    auto read_targets = [&](int (&target)[FM]) __attribute__((always_inline)) {
        if constexpr (XENT) {
            const uint32_t at = lds_base + kStages * STAGE + which * TGB + (wr * WTM + (lane_id() & 15)) * 8;
            tg_u32x2 v[FM];
#pragma unroll
            for (int i = 0; i < FM; ++i)
                asm volatile("ds_read_b64 %0, %1 offset:%2" : "=v"(v[i]) : "v"(at), "i"(i * 128));
            __builtin_amdgcn_s_waitcnt(WAIT_VM_LGKM0(63));
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                asm volatile("" : "+v"(v[i]));
                target[i] = v[i].y == 0 ? (int)v[i].x : -1;
            }
        }
    };

    const float alpha = PLAIN ? read_alpha(L) : 1.0f;
    Tile cu, nx{};
    int slot = seek(blockIdx.x, cu);
    if (slot < 0) return;
    load_targets(cu, 0);
    stream(cu, true);
#pragma unroll
    for (int s = 0; s < kStages; s += SPL) {
        open_stage();
#pragma unroll
        for (int y = 0; y < LPS; ++y) gload(s * STAGE, y);
        close_stage();
    }
    __builtin_amdgcn_s_waitcnt(WAIT_VM_LGKM0(kStages / SPL * LPS - LPS));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    for_each(std::make_integer_sequence<int, FM + FN>{},
             [&](auto Y) __attribute__((always_inline)) { read(0, 0, Y); });
    __builtin_amdgcn_s_waitcnt(WAIT_VM_LGKM0((kStages - 2) * LPS));
    __builtin_amdgcn_sched_barrier(0);
    tie(0);
    for (;;) {
        const int nslot = seek(slot + grid, nx);
        const bool more = nslot >= 0;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = tg_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        // (from stage kStages before the end on, the loads are the next tile's
        // first ones, or zeros)
#pragma clang loop unroll(disable)
        for (int kt = cu.stages; kt > 0; kt -= 2) {
            // (past this tile's first barrier: nobody reads the last tile's
            // targets any more, whose buffer takes the next one's)
            if (XENT && more && kt == cu.stages - 2) load_targets(nx, which ^ 1);
            if (kStages % 2 == 0 && kt == kStages) stream(more ? nx : cu, more);
            body(std::integral_constant<int, 0>{});
            if (kStages % 2 == 1 && kt == kStages + 1) stream(more ? nx : cu, more);
            body(std::integral_constant<int, 1>{});
        }
        if (cu.split >= 0) {
            keep_part<FM, NW>(L, cu.t - L.whole, cu.split, wave, acc);
        } else {
            int target[FM];
            read_targets(target);
            finish<EPI, BKM, FM>(L, cu.prob, alpha, acc, cu.m0 + wr * WTM, cu.n0 + wc * (GLU ? 32 : 64), target);
        }
        which ^= 1;
        if (!more) break;
        cu = nx;
        slot = nslot;
    }
    // the loads past the last tile write zeros to LDS: they end before it does
    __builtin_amdgcn_s_waitcnt(0);
}

// The tiles that were split: their parts' sums, added in order, and then what
// the whole tiles' workgroups do.  A wave takes 16 rows of what one wave of
// the tile held (four a workgroup, each on its own), so that few tiles still
// fill the GPU.
template <int TILE, int EPI, bool BKM>
__global__ __launch_bounds__(256) void tg_join_kernel(TgLaunch L) {
    using C = Cfg<TILE>;
    constexpr int NW = C::WR * C::WC, WTM = C::BM / C::WR, FM = WTM / 16;
    constexpr bool GLU = EPI == kTgGlu || EPI == kTgGluBack;
    const int lane = threadIdx.x & 63;
    const int id = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    const int rt = id / (NW * FM), wave = id / FM % NW, i = id % FM;
    if (rt >= L.tiles - L.whole) return;
    const tg_f32x4 *p = reinterpret_cast<const tg_f32x4 *>(L.part) +
                        (((int64_t)rt * L.splits * NW + wave) * FM + i) * (4 * 64) + lane;
    tg_f32x4 acc[1][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[0][j] = p[j * 64];
#pragma unroll 4
    for (int s = 1; s < L.splits; ++s) {
        p += (int64_t)NW * FM * (4 * 64);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[0][j] += p[j * 64];
    }
    const int t = L.whole + rt, per = L.tiles_m * L.tiles_n, prob = t >= per ? 1 : 0;
    int ti, tj;
    tile_at(t - prob * per, L.tiles_m, L.tiles_n, ti, tj);
    const int R0 = ti * C::BM + (wave / C::WC) * WTM + i * 16;
    int target[1] = {-1};
    if constexpr (EPI == kTgXent) {
        const int row = R0 + (lane & 15);
        const int64_t v = row < L.M ? L.target[row] : -1;
        if (v >= 0 && v <= 0x7FFFFFFF) target[0] = (int)v;
    }
    finish<EPI, BKM, 1>(L, prob, read_alpha(L), acc, R0, tj * (GLU ? C::BN / 2 : C::BN) + (wave % C::WC) * (GLU ? 32 : 64), target);
}

// Compute units of the current device (asked for once), a multiple of the 8
// XCDs.
int compute_units() {
    static const int cus = [] {
        int dev = 0, n = 0;
        if (hipGetDevice(&dev) != hipSuccess ||
            hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 8)
            n = 256;
        return n / 8 * 8;
    }();
    return cus;
}

template <int TILE, int EPI, bool AKM, bool BKM>
hipError_t run(TgLaunch &L, hipStream_t stream) {
    using C = Cfg<TILE>;
    constexpr bool GLU = EPI == kTgGlu || EPI == kTgGluBack;
    constexpr int BO = GLU ? C::BN / 2 : C::BN, threads = C::WR * C::WC * 64;
    L.tiles_m = (L.M + C::BM - 1) / C::BM;
    L.tiles_n = (L.N + BO - 1) / BO;
    const int64_t tiles = (int64_t)L.tiles_m * L.tiles_n * L.nprob;
    const int64_t total = L.whole + (tiles - L.whole) * L.splits;
    if (tiles > 0x7FFFFF00 || total > 0x7FFFFF00) return hipErrorInvalidValue;
    L.tiles = (int32_t)tiles;
    L.total = (int32_t)total;
    L.padded = (L.total + 7) / 8 * 8;
    const int64_t round = (int64_t)compute_units() * (C::WPE * 4 / (threads / 64));
    const uint32_t grid = (uint32_t)(L.padded < round ? L.padded : round);
    hipLaunchKernelGGL((tg_kernel<TILE, EPI, AKM, BKM>), dim3(grid + ((EPI == kTgStore || EPI == kTgSum) && L.sum_up.loss != nullptr ? 1 : 0)),
                       dim3(threads), 0, stream, L);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && L.splits > 1) {
        const int64_t waves = (tiles - L.whole) * (C::BM / 16) * C::WC;
        hipLaunchKernelGGL((tg_join_kernel<TILE, EPI, BKM>), dim3((uint32_t)((waves + 3) / 4)), dim3(256), 0, stream, L);
        e = hipGetLastError();
    }
    return e;
}

template <int EPI, bool AKM, bool BKM>
hipError_t run_tile(TgLaunch &L, hipStream_t stream) {
    if (L.tile == kTile256) return run<kTile256, EPI, AKM, BKM>(L, stream);
    if (L.tile == kTile256x128) return run<kTile256x128, EPI, AKM, BKM>(L, stream);
    if (L.tile == kTile128) return run<kTile128, EPI, AKM, BKM>(L, stream);
    return run<kTile64, EPI, AKM, BKM>(L, stream);
}

}  // namespace

// Tile and split, by an estimate of the launch's time in microseconds from
// figures measured on the card (256 CUs):
//   stage   one workgroup alone on its CU takes `alone` a stage of 32, bound by
//           latency; a CU with all it holds (`held` of them) held * across, or
//           held * along with both operands row-major (256 x 128 tiles, whose
//           three buffers hold no pairs of stages, load halves of lines then)
//   tile    its first loads and its epilogue: `plain`, or `heavy` with
//           exponentials
//   split   a second launch (4) and 8 bytes an output and part at 5 TB/s
// Full rounds of tiles are computed whole; those left over, which would leave
// CUs idle, may be split along the reduction: [256, 50304] x [50304, 768]
// takes 937 us whole on 256 x 256 tiles, 54 us in 16 parts on 128 x 128, 39 us in
// the 21 parts that this chooses.
// Over 70 calls of drawn sizes each forced to one kind of tile, the choice took
// at most 5% longer than the best of the four but for six (6 to 13%, all but
// one of them under 100 us).
void plan_tg(TgEpilogue epi, TgLaunch &L) {
    struct Figures {
        int tile, bm, bn, held;
        double alone, across, along, plain, heavy;
    };
    static constexpr Figures figures[4] = {{kTile256, 256, 256, 1, 0.66, 0.86, 0.80, 4.0, 10.0},
                                           {kTile256x128, 256, 128, 2, 0.46, 0.485, 0.60, 3.0, 8.0},
                                           {kTile128, 128, 128, 2, 0.27, 0.25, 0.28, 2.0, 7.0},
                                           {kTile64, 64, 64, 4, 0.17, 0.13, 0.12, 1.5, 6.0}};
    constexpr int64_t cus = 256;  // (the figures' card; a launch takes the device's own count)
    const bool glu = epi == kTgGlu || epi == kTgGluBack;
    int all = L.prob[0].seg[0].stages;
    if (!glu && L.prob[0].nseg > 1) all += L.prob[0].seg[1].stages;
    double best = 0;
    for (const Figures &f : figures) {
        const int64_t bn = glu ? f.bn / 2 : f.bn, held = f.held * cus;
        const int64_t tiles = (L.M + f.bm - 1) / f.bm * ((L.N + bn - 1) / bn) * L.nprob;
        const int64_t rounds = tiles / held, rest = tiles % held;
        const bool plain = epi == kTgStore || epi == kTgSum;
        const double each = plain ? f.plain : f.heavy, busy = plain ? f.across : f.along;
        auto load = [&](int64_t n) {
            // (one on each of few CUs is not held up by the others; nor, across
            // lines, one where two would fit)
            const bool few = n == 1 && ((plain && f.held > 1) || tiles < cus / 2);
            return few || f.alone > n * busy ? f.alone : n * busy;
        };
        const double whole = rounds * (all * load(f.held) + each);
        for (int split = 1; split <= 32; ++split) {
            const int per = (all / 2 + split - 1) / split * 2;
            if (split > 1 && (per < 8 || rest == 0)) break;
            if ((all + per - 1) / per != split) continue;
            const int64_t on = (rest * split + cus - 1) / cus, full = on / f.held, left = on % f.held;
            double t = whole + full * (per * load(f.held) + each) + (left ? per * load(left) + each : 0.0);
            if (split > 1) t += 4.0 + 8.0 * split * (double)(rest * f.bm * f.bn) / 5.0e6;
            if (best == 0 || t < best) {
                best = t;
                L.tile = f.tile;
                L.splits = split;
                L.split_stages = per;
                L.whole = (int32_t)(split > 1 ? tiles - rest : tiles);
            }
        }
    }
    L.ldsum = (L.N + 3) / 4 * 4;
}

size_t tg_part_bytes(TgEpilogue epi, const TgLaunch &L) {
    if (L.splits == 1) return 0;
    const int64_t bm = L.tile == kTile64 ? 64 : L.tile == kTile128 ? 128 : 256;
    const int64_t bn = L.tile == kTile256x128 ? 128 : bm, bo = epi == kTgGlu || epi == kTgGluBack ? bn / 2 : bn;
    const int64_t tiles = (L.M + bm - 1) / bm * ((L.N + bo - 1) / bo) * L.nprob;
    return (size_t)((tiles - L.whole) * L.splits * bm * bn * 4);
}

hipError_t launch_tg(TgEpilogue epi, bool a_km, bool b_km, TgLaunch &L, hipStream_t stream) {
    if (epi == kTgXent) return run_tile<kTgXent, false, false>(L, stream);
    if (epi == kTgGlu) return run_tile<kTgGlu, false, false>(L, stream);
    if (epi == kTgGluBack) return run_tile<kTgGluBack, false, false>(L, stream);
    if (!b_km || (epi == kTgSum && !a_km)) return hipErrorInvalidValue;
    if (epi == kTgSum) return run_tile<kTgSum, true, true>(L, stream);
    return a_km ? run_tile<kTgStore, true, true>(L, stream) : run_tile<kTgStore, false, true>(L, stream);
}

}  // namespace zopt
