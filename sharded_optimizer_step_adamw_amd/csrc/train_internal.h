// train_internal.h -- declarations shared by the operators that produce a
// rank's gradients: linear cross entropy, the gated feed-forward block and
// 8-bit activation checkpoints (train_gemm.hip, train_rows.hip, train_api.hip).
#pragma once

#include "zopt_internal.h"

namespace zopt {

// ------------------------------------------------------- matrix products
//
// C[M x N] = sum over segments of A B^T.  Each operand is a 16-bit matrix
// whose contiguous side is a multiple of 8 elements, as are its row stride
// and its base's alignment (operands that are not are copied into the
// workspace first); outer is the side that indexes C (M or N), k the reduction.
//   row-major  [outer, k]   (k contiguous)
//   k-major    [k, outer]   (outer contiguous)
// Everything outside outer x k reads as zero.
struct TgOperand {
    const uint16_t *p;
    int64_t ld;        // elements between rows, < 2^22
    int32_t outer, k;  // extents
};

struct TgSegment {
    TgOperand a, b;
    int32_t stages;    // max(a.k, b.k) / 32, up to an even number
};

// What becomes of a tile:
//   kTgStore    alpha * sum -> bf16
//   kTgSum      the same with fp32 sums kept between calls (see below)
//   kTgXent     exponentials and row statistics of a piece of logits
//   kTgGlu      act(g) u from interleaved gate / up columns, with checkpoints
//   kTgGluBack  dg, du (and h) from g, u and dh
//   kTgFloat    sum -> fp32
//   kTgMoeBack  kTgGluBack for rows with a weight each, from fp32 dh, with the
//               weights' gradients
//   kTgRows     sum -> fp16 with a power of two per row and 64 columns
enum TgEpilogue : int {
    kTgStore = 0, kTgXent = 1, kTgGlu = 2, kTgGluBack = 3, kTgSum = 4, kTgFloat = 5, kTgMoeBack = 6, kTgRows = 7
};

// Products of several groups (experts) in one launch, whose sizes only the
// device knows: a group's rows are some neighbouring ones of the operands that
// the groups share.
//   kGroupRows   those are rows of A and of the output; each group has a B
//                (B's p, and groups' distance group_stride)
//   kGroupDepth  those are the reduction of A and B; each group has an output
//                (out, and group_out)
enum TgGroups : int { kNoGroups = 0, kGroupRows = 1, kGroupDepth = 2 };
// What a gathered operand spans at most (its offsets are 32 bits wide).
constexpr int64_t kGatherBytes = 0xFFFF0000ll;
// A tile row of kGroupRows: its group, its first row and the group's last.
// The list's first entry holds the number of the others (in `group`).
struct TgTileRow {
    int32_t group, row, end, unused;
};
// What a tile of kGroupDepth sums over: rows row .. end - 1 of a group, all of
// them or, of a group with more than part_rows, a part.  The list's first entry
// holds the number of items (in `group`), of those that are parts, which come
// first (in `row`), and of the groups that have parts (in `end`); `joins` lists
// those: the group, its first item, the item behind its last.
typedef TgTileRow TgItem;

enum TgAct : int { kActSilu = 0, kActGelu = 1 };

struct TgProblem {
    TgSegment seg[2];
    int32_t nseg;
    uint16_t *out;     // bf16 [M, N], row stride ldc
    float *sum;        // fp32 [M, N] (row stride ldsum), or NULL
};

// The loss from its rows: share * sum, share = 1 or (mean) 1 / the rows whose
// target is not `ignore` (0 if none).
struct TgTotal {
    const float *row_loss;
    const int64_t *target;
    int64_t rows, ignore;
    int32_t mean;
    float *loss;
};

struct TgLaunch {
    TgProblem prob[2];
    int32_t nprob;
    int32_t M, N;             // output sizes (Glu: N = feed-forward width)
    int32_t tile, tiles_m, tiles_n;  // kind of tile, grid of output tiles
    // Tiles [0, whole) are computed in one go, the others in `splits` parts of
    // split_stages stages each, kept in `part` (fp32) and joined by a second
    // launch
    int32_t whole, splits, split_stages;
    int32_t tiles, total, padded;  // tiles of all problems; with parts; rounded up to 8
    float *part;
    int64_t ldc;
    // kTgStore, kTgSum
    const float *alpha;       // device scalar, or NULL: 1
    // kTgSum
    int64_t ldsum;
    int32_t sum_in, sum_out;  // add prob.sum first; write fp32 to prob.sum (else bf16 to out)
    TgTotal sum_up;           // loss not NULL: one more workgroup forms it
    // kTgXent: e [M, lde] fp16 (NULL: statistics only), per row r and 64-column
    // group g stats[r * ldstat + g] = (max, sum of exponentials); the target's
    // logit to zt
    uint16_t *e;
    int64_t lde;
    int32_t past;             // e is written past the caches
    float2 *stats;
    int64_t ldstat;
    const int64_t *target;
    float *zt;
    // kTgGlu / kTgGluBack (row strides: h ldc; q F bytes; scale ceil(F / 32); dh lddh; dg, du lddg)
    int32_t act;
    uint16_t *h;              // kTgGluBack: may be NULL
    uint8_t *g8, *u8;         // checkpoint values, or NULL
    uint8_t *gs, *us;
    const uint16_t *dh;
    int64_t lddh;
    uint16_t *dg, *du;        // row stride lddg, columns [N, round up to 8) written as zero
    int64_t lddg;
    // kTgMoeBack: h is share * act(g) u, dg and du are of share * dh (their strides
    // lddg, as h's); dot [M, lddot]: the sums of dh act(g) u over 32 columns
    const float *dhf;         // fp32, row stride lddh, columns [N, round up to 4) readable
    const float *share;       // [M]
    float *dot;
    int64_t lddot;
    // kTgRows: values to prob.out, exponents to row_scale [M, ldscale] (see tg_rows_*)
    uint8_t *row_scale;
    int64_t ldscale;
    // groups (whole, tiles, total and padded are the kernel's own)
    const TgTileRow *tile_row;  // kGroupRows; NULL: from offsets [groups + 1] (64 groups at most)
    const int32_t *offsets;
    const TgItem *items, *joins;
    int32_t item_limit, join_limit;  // no more than that many; join_limit 0: no parts
    int32_t part_rows;        // a multiple of 64
    int32_t groups, slots;    // (rows of all groups)
    // gathered A (kGroupRows): row r is row order[r] / top of the operand, which has
    // `tokens` (an order that is no slot: a row of zeros).  The quotient of s < 2^30 by
    // top <= 2^k is s times top_times = ceil(2^(31 + k) / top), over 2^(31 + k): too
    // large by less than s 2^k / (2^(31 + k) top) < 1 / top.
    const int32_t *order;
    int32_t tokens, top_shift;
    uint32_t top_times;
    void set_top(int32_t top) {
        top_shift = 0;
        while ((1 << top_shift) < top) ++top_shift;
        top_times = (uint32_t)((((uint64_t)1 << (31 + top_shift)) + top - 1) / top);
    }
    int64_t group_stride, group_out;
};

constexpr int kXentGroup = 64;  // columns per statistics group

// Chooses tile and split (sets tile, whole, splits, split_stages, ldsum) from
// the sizes, problems and segments; the parts' fp32 scratch.
void plan_tg(TgEpilogue epi, TgLaunch &L);
size_t tg_part_bytes(TgEpilogue epi, const TgLaunch &L);

// a_km / b_km: operand is k-major.  kTgXent and the Glu kinds: both row-major;
// kTgSum: both k-major; kTgStore: b k-major.
hipError_t launch_tg(TgEpilogue epi, bool a_km, bool b_km, TgLaunch &L, hipStream_t stream);

// ------------------------------------------------------------- row passes

// The memory-side cache of 256 MiB serves a pass what the pass before wrote if
// that fits it.  Where a matrix does not, or would push out what the next
// pass needs, its accesses go past the caches.
constexpr int64_t kCacheBytes = (int64_t)256 << 20;

// What a call does to its operands before its products, all in one launch:
//   kPrepCopy    dst [rows, round8(cols)] = src [rows, cols] (row stride ld), zero
//                beyond cols and in rows whose target is `ignore` (target NULL: none)
//   kPrepUnpack  dst [rows, round8(cols)] = the values of the checkpoint q, scale
//   kPrepBack    dst = dg, dst2 = du (row stride dst_ld, zero in columns [cols,
//                round8(cols))) and h (or NULL, row stride h_ld) from the
//                checkpoint q, scale of g and q2, scale2 of u and from src = dh
//   kPrepCount   *factor = grad_scale, or (mean) grad_scale / rows that take part (0
//                if none)
enum TgPrepKind : int { kPrepCopy = 0, kPrepUnpack = 1, kPrepBack = 2, kPrepCount = 3 };
struct TgPrep {
    int32_t kind, act, mean;
    uint32_t blocks;          // set by the launch
    int64_t rows, cols;
    const uint16_t *src;
    int64_t ld;
    const uint8_t *q, *scale, *q2, *scale2;
    uint16_t *dst, *dst2, *h;
    int64_t dst_ld, h_ld;
    const int64_t *target;
    int64_t ignore;
    float grad_scale;
    float *factor;
};
constexpr int kMaxPreps = 4;
struct TgPrepList {
    TgPrep job[kMaxPreps];
    int32_t n;
};
hipError_t launch_prep(TgPrepList &list, hipStream_t stream);
hipError_t launch_fill_zero(uint16_t *dst, int64_t ld, int64_t rows, int64_t cols,
                            hipStream_t stream);

hipError_t launch_act8_pack(const uint16_t *x, int64_t ld, int64_t rows, int64_t cols, uint8_t *q,
                            uint8_t *scale, hipStream_t stream);
hipError_t launch_act8_unpack(const uint8_t *q, const uint8_t *scale, int64_t rows, int64_t cols,
                              uint16_t *x, int64_t ld, hipStream_t stream);

// Rows [0, rows): row losses from the group statistics [rows, groups] and the
// targets' logits; with e (fp16 exponentials, row stride lde) also P = softmax
// - onehot (bf16) in its place, columns [V, lde) zero.
hipError_t launch_xent_rows(const float2 *stats, int32_t groups, const int64_t *target,
                            int64_t ignore, int32_t V, const float *zt, int64_t rows,
                            float *row_loss, uint16_t *e, int64_t lde, bool past,
                            hipStream_t stream);
hipError_t launch_xent_total(const TgTotal &t, hipStream_t stream);

// ---------------------------------------------------------- device helpers

// The number of rows that take part, summed over a block of N threads.
template <int N>
__device__ __forceinline__ long long tg_valid_rows(const int64_t *__restrict__ target, int64_t rows,
                                                   int64_t ignore) {
    __shared__ long long part[N / 64];
    long long n = 0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < rows; i += N) n += target[i] != ignore ? 1 : 0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = n;
    __syncthreads();
    long long all = 0;
    for (int k = 0; k < N / 64; ++k) all += part[k];
    return all;
}
__device__ __forceinline__ double tg_share(long long rows, int mean) {
    return !mean ? 1.0 : rows > 0 ? 1.0 / (double)rows : 0.0;
}
// the loss from its rows by a block of N threads: in double, in a fixed order
template <int N>
__device__ __forceinline__ void tg_total(const TgTotal &t) {
    __shared__ double part[N / 64];
    const long long n = t.mean ? tg_valid_rows<N>(t.target, t.rows, t.ignore) : 0;
    double s = 0.0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < t.rows; i += N) s += (double)t.row_loss[i];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0.0;
        for (int k = 0; k < N / 64; ++k) all += part[k];
        *t.loss = (float)(all * tg_share(n, t.mean));
    }
}

// two fp32 -> two bf16 / fp16, round to nearest even, one instruction each; a
// NaN stays a NaN
typedef __bf16 tg_bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 tg_f16x2 __attribute__((ext_vector_type(2)));
typedef float tg_f32x2 __attribute__((ext_vector_type(2)));
typedef float tg_f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t tg_u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t tg_u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t tg_pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(tg_f32x2{lo, hi}, tg_bf16x2));
}
__device__ __forceinline__ tg_u32x4 tg_pack8(const float (&v)[8]) {
    return tg_u32x4{tg_pack_bf16(v[0], v[1]), tg_pack_bf16(v[2], v[3]), tg_pack_bf16(v[4], v[5]),
                    tg_pack_bf16(v[6], v[7])};
}
__device__ __forceinline__ void tg_unpack8(tg_u32x4 p, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(p[k] << 16);
        v[2 * k + 1] = __uint_as_float(p[k] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint32_t tg_pack_f16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(tg_f32x2{lo, hi}, tg_f16x2));
}

// An activation's value and derivative.  silu(g) = g s(g) with the logistic
// s; gelu's tanh form is g s(y), y = sqrt(8 / pi) (g + 0.044715 g^3), since
// (1 + tanh(y / 2)) / 2 = s(y).
struct TgActValue {
    float a, da;
};
__device__ __forceinline__ TgActValue tg_act(float g, int32_t act) {
    float y = g, dy = 1.0f;
    if (act == kActGelu) {
        // (beyond +-16 s is 1 or 0 to every bit and s (1 - s) is 0; the polynomials
        // end there, since an infinite dy times that 0 would be NaN)
        const float k = 1.5957691216057308f, b = __builtin_amdgcn_fmed3f(g, -16.0f, 16.0f);
        const float g2 = b * b;
        y = k * (b + 0.044715f * (g2 * b));
        dy = k * (1.0f + 0.134145f * g2);
    }
    const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-y));
    return {g * s, s + g * (s * (1.0f - s)) * dy};
}

// The 8-bit checkpoint's scale byte from the bit pattern of a block's largest
// magnitude (as an integer, so NaN > Inf > finite): the smallest power of two
// 2^(byte - 127) with amax <= 448 * 2^(byte - 127), 448 = 1.75 * 2^8 being
// e4m3's largest value, and at least 2^-124, below which a product with
// e4m3's subnormals would leave bf16's; 255 if a value is not finite.
__device__ __forceinline__ uint32_t tg_scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7F800000u) return 255u;
    const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return e < 3 ? 3u : (uint32_t)e;
}
// 2^(127 - byte), what values are multiplied with (NaN for byte 255), and
// 2^(byte - 127), what they are read back with
__device__ __forceinline__ float tg_scale_in(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float tg_scale_out(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23);
}
// Rows of sums that a later pass adds up, in 16 bits: fp16 times 2^(exponent -
// 141), one exponent for 64 neighbouring columns, that of the largest finite value
// there (at least 14), which so lies in [2^14, 2^15) of fp16.  The rounding is off
// by 2^-11 of a value, where bf16's 2^-8 would be as much as that of the result
// itself, or by 2^-39 of the largest.  (fp32 rows would double the bytes of two
// passes that HBM bounds.)
constexpr int kRowsGroup = 64;
__device__ __forceinline__ uint32_t tg_finite_bits(float v) {
    const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
    return b < 0x7F800000u ? b : 0u;
}
__device__ __forceinline__ uint32_t tg_rows_exponent(uint32_t largest_bits) {
    const uint32_t e = largest_bits >> 23;
    return e < 14 ? 14u : e;
}
__device__ __forceinline__ float tg_rows_in(uint32_t exponent) { return __uint_as_float((268u - exponent) << 23); }
__device__ __forceinline__ float tg_rows_out(float v, uint32_t exponent) {
    return __builtin_amdgcn_ldexpf(v, (int)exponent - 141);
}

// Eight fp32 -> eight e4m3 of v * 2^(127 - byte), round to nearest even, low
// first.  At the topmost scale, 2^120, 240 is the largest code: the next one,
// 256, stands for 2^128, which no bf16 holds (and 240 is within 2^-4 of every
// value up to the largest fp32).
__device__ __forceinline__ tg_u32x2 tg_pack_e4m3(const float (&x)[8], uint32_t byte) {
    const float s = tg_scale_in(byte), top = byte == 247u ? 240.0f : 448.0f;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __builtin_amdgcn_fmed3f(x[k] * s, -top, top);
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
    return tg_u32x2{(uint32_t)lo, (uint32_t)hi};
}
__device__ __forceinline__ void tg_unpack_e4m3(tg_u32x2 q, float s, float (&v)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int w = (int)(h ? q.y : q.x);
        const tg_f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
        const tg_f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
        v[4 * h + 0] = a.x * s;
        v[4 * h + 1] = a.y * s;
        v[4 * h + 2] = b.x * s;
        v[4 * h + 3] = b.y * s;
    }
}

// 8 and 16 bytes at any address (global memory takes them unaligned)
template <class V>
__device__ __forceinline__ V tg_load(const void *p) {
    V v;
    __builtin_memcpy(&v, p, sizeof v);
    return v;
}
template <class V>
__device__ __forceinline__ void tg_store(void *p, V v) {
    __builtin_memcpy(p, &v, sizeof v);
}
// ... past the caches (PAST), for data that is not met again before the
// memory-side cache has seen more than it holds
template <class V, bool PAST>
__device__ __forceinline__ V tg_load(const void *p) {
    typedef V U __attribute__((aligned(1)));
    if constexpr (PAST)
        return __builtin_nontemporal_load(reinterpret_cast<const U *>(p));
    else
        return tg_load<V>(p);
}
template <bool PAST, class V>
__device__ __forceinline__ void tg_store(void *p, V v) {
    typedef V U __attribute__((aligned(1)));
    if constexpr (PAST)
        __builtin_nontemporal_store(v, reinterpret_cast<U *>(p));
    else
        tg_store(p, v);
}
// up to 8 bytes / 16-bit values at p, of which the first n exist
__device__ __forceinline__ tg_u32x2 tg_load8b(const uint8_t *p, int n) {
    if (n >= 8) return tg_load<tg_u32x2>(p);
    tg_u32x2 r{0, 0};
    for (int k = 0; k < 8; ++k)
        if (k < n) {
            if (k < 4) r.x |= (uint32_t)p[k] << (8 * k);
            else r.y |= (uint32_t)p[k] << (8 * (k - 4));
        }
    return r;
}
__device__ __forceinline__ void tg_store8b(uint8_t *p, tg_u32x2 v, int n) {
    if (n >= 8) {
        tg_store(p, v);
        return;
    }
    for (int k = 0; k < 8; ++k)
        if (k < n) p[k] = (uint8_t)((k < 4 ? v.x >> (8 * k) : v.y >> (8 * (k - 4))) & 0xFFu);
}
template <bool PAST = false>
__device__ __forceinline__ tg_u32x4 tg_load8h(const uint16_t *p, int n) {
    if (n >= 8) return tg_load<tg_u32x4, PAST>(p);
    tg_u32x4 r{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < n) r[k >> 1] |= (uint32_t)p[k] << (16 * (k & 1));
    return r;
}
template <bool PAST = false>
__device__ __forceinline__ void tg_store8h(uint16_t *p, tg_u32x4 v, int n) {
    if (n >= 8) {
        tg_store<PAST>(p, v);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < n) p[k] = (uint16_t)((v[k >> 1] >> (16 * (k & 1))) & 0xFFFFu);
}

}  // namespace zopt
