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
#include "train_internal.h"

namespace zopt {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

#define LDS_ADDR(p) ((__attribute__((address_space(3))) void *)(p))

constexpr int kBK = 32;  // reduction elements per stage

// Tile t of a tiles_m x tiles_n grid.
__device__ __forceinline__ void tile_at(int t, int tm, int tn, int &ti, int &tj) {
    ti = t % tm;
    tj = t / tm;
}

// Row statistics and exponentials of a logits tile.  A wave's 64 columns are
// one statistics group: m = their largest logit, s = the sum of exp(z - m),
// and e = exp(z - m) in (0, 1] kept in fp16 (11 bits; what is lost below
// 2^-14 is under 2^-25 of the group's largest).
template <int FM>
__device__ __forceinline__ void xent_epilogue(const TgLaunch &L, tg_f32x4 (&acc)[FM][4], int R0, int C0,
                                              int lane) {
    const int c = lane & 15, q = lane >> 4;
    if (C0 >= (int)L.lde && C0 >= L.N) return;
    const int64_t group = C0 / kXentGroup;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int row = R0 + i * 16 + c;
        float z[16];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int col = C0 + h * 32 + q * 8 + k;
                z[h * 8 + k] = col < L.N ? acc[i][2 * h + (k >> 2)][k & 3] : -INFINITY;
            }
        float m = z[0];
#pragma unroll
        for (int k = 1; k < 16; ++k) m = fmaxf(m, z[k]);
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        if (row < L.M) {
            const int64_t t = L.target[row];
            const int64_t rel = t - C0 - q * 8;
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (rel == (k >> 3) * 32 + (k & 7)) L.zt[row] = z[k];
        }
        // a group of -inf alone: exponentials 0, not NaN
        const float ref = m == -INFINITY ? 0.0f : m;
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            z[k] = __expf(z[k] - ref);
            s += z[k];
        }
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (row < L.M) {
            if (q == 0 && C0 < L.N) L.stats[group * L.ldstat + row] = make_float2(m, s);
            if (L.e != nullptr) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int col = C0 + h * 32 + q * 8;
                    if (col < L.lde)
                        *reinterpret_cast<tg_u32x4 *>(L.e + (int64_t)row * L.lde + col) =
                            tg_u32x4{tg_pack_f16(z[8 * h], z[8 * h + 1]), tg_pack_f16(z[8 * h + 2], z[8 * h + 3]),
                                     tg_pack_f16(z[8 * h + 4], z[8 * h + 5]),
                                     tg_pack_f16(z[8 * h + 6], z[8 * h + 7])};
                }
            }
        }
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
                                           int q, bool live, bool vec) {
    uint32_t big = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t b = __float_as_uint(v[k]) & 0x7FFFFFFFu;
        big = k < n && b > big ? b : big;
    }
    uint32_t o = __shfl_xor(big, 16);
    big = o > big ? o : big;
    o = __shfl_xor(big, 32);
    big = o > big ? o : big;
    const uint32_t byte = tg_scale_byte(big);
    if (!live) return;
    if (n > 0) tg_store8b(qrow + col, tg_pack_e4m3(v, byte), n, vec);
    if (q == 0) srow[col >> 5] = (uint8_t)byte;
}

// Gate and up columns of a tile: blocks 0, 1 are the gate's 32 columns, 2, 3
// the up projection's same columns; C0 is the first of them.
template <int FM, bool BACK>
__device__ __forceinline__ void glu_epilogue(const TgLaunch &L, tg_f32x4 (&acc)[FM][4], int R0, int C0, int lane) {
    const int c = lane & 15, q = lane >> 4;
    const int F = L.N;
    if (C0 >= F) return;
    const int col = C0 + q * 8;
    const int n = F - col > 8 ? 8 : F - col < 0 ? 0 : F - col;
    const int64_t blocks = (F + 31) / 32;
    const bool vec = L.vec != 0, qvec = (F & 7) == 0;
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
            if (live && n > 0) tg_store8h(L.h + (int64_t)row * L.ldc + col, pack8(h), n, vec);
            if (L.g8 != nullptr) {
                act8_store(g, n, L.g8 + (int64_t)row * F, L.gs + (int64_t)row * blocks, col, q, live, qvec);
                act8_store(u, n, L.u8 + (int64_t)row * F, L.us + (int64_t)row * blocks, col, q, live, qvec);
            }
        } else {
            if (live && n > 0) {
                float dh[8], dg[8], du[8];
                unpack8(tg_load8h(L.dh + (int64_t)row * L.lddh + col, n, L.dhvec != 0), dh);
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
                if (L.h != nullptr) tg_store8h(L.h + (int64_t)row * L.ldc + col, pack8(h), n, vec);
            }
        }
    }
}

// A tile of sums: alpha * acc to bf16, or fp32 sums kept for a later call.
// PERM: the column order of a row-major B (eight consecutive per lane).
template <int FM, int FN, bool PERM>
__device__ __forceinline__ void store_epilogue(const TgLaunch &L, const TgProblem &P, tg_f32x4 (&acc)[FM][FN],
                                               int R0, int C0, int lane) {
    const int c = lane & 15, q = lane >> 4;
    const float alpha = L.alpha ? *L.alpha : 1.0f;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int row = R0 + i * 16 + c;
        if (row >= L.M) continue;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int col = C0 + (PERM ? (j >> 1) * 32 + q * 8 + (j & 1) * 4 : j * 16 + q * 4);
            if (col >= L.N) continue;
            tg_f32x4 v = acc[i][j];
            if (L.sum_in || L.sum_out) {
                // (rows of fp32 sums are padded to a multiple of 4)
                tg_f32x4 *s = reinterpret_cast<tg_f32x4 *>(P.sum + (int64_t)row * L.ldsum + col);
                if (L.sum_in) v += *s;
                if (L.sum_out) {
                    *s = v;
                    continue;
                }
            }
            uint16_t *o = P.out + (int64_t)row * L.ldc + col;
            const tg_u32x2 p{tg_pack_bf16(v[0] * alpha, v[1] * alpha), tg_pack_bf16(v[2] * alpha, v[3] * alpha)};
            if (L.vec && col + 4 <= L.N) {
                *reinterpret_cast<tg_u32x2 *>(o) = p;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (col + k < L.N) o[k] = (uint16_t)((k < 2 ? p.x : p.y) >> (16 * (k & 1)));
            }
        }
    }
}

// One BM x BM output tile per workgroup of WR x 2 waves, each BM / WR x 64
// columns from 16 x 16 x 32 MFMAs with fp32 accumulators.  Stages of 32
// reduction elements go from global memory straight to LDS, 16 bytes a lane;
// a lane outside the operand reads past the buffer descriptor's end, which
// gives zeros.  LDS layouts (as in the Newton-Schulz kernels): row-major rows
// of 64 bytes, 16-byte chunk c of row r at slot c ^ ((r >> 1) & 3); k-major
// rows of 2 BM bytes, 32-byte unit u of row r at unit u ^ qsw(r).
template <int BM, int EPI, bool AKM, bool BKM>
__global__ __launch_bounds__(256) void tg_kernel(TgLaunch L) {
    constexpr int NW = 4, WC = 2, WR = 2, WTM = BM / WR, WTN = BM / WC, FM = WTM / 16, FN = WTN / 16;
    static_assert(WTN == 64, "a wave holds 64 columns");
    constexpr int ROW = 64, OPB = BM * ROW, LOADS = OPB / 1024 / NW;
    constexpr int QRB = 2 * BM, QCH = QRB / 16;
    constexpr bool GLU = EPI == kTgGlu || EPI == kTgGluBack;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * OPB];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave / WC, wc = wave % WC;
    const uint32_t lds_base = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t *)lds);

    const int per = L.tiles_m * L.tiles_n;
    const int pi = blockIdx.x / per;
    const TgProblem &P = L.prob[pi];
    int ti, tj;
    tile_at(blockIdx.x - pi * per, L.tiles_m, L.tiles_n, ti, tj);
    // gate / up tiles hold BM / 2 columns of each
    const int m0 = ti * BM, n0 = tj * (GLU ? BM / 2 : BM);

    auto qsw = [](int r) __attribute__((always_inline)) {
        return BM >= 128 ? (r & 3) | (((r >> 3) & 1) << 2) : ((r >> 1) & 1) | (((r >> 3) & 1) << 1);
    };

    tg_f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = tg_f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // kilobyte kb of an operand's stage: 16 rows (row-major), or 1024 / QRB
    // k rows; the lane's byte offset from the stage's corner
    auto load_rows = [&](const TgOperand &o, const uint16_t *base, int left, int k0, int kb, int row, int dst)
                         __attribute__((always_inline)) {
        // left: rows of the operand from the tile's first one on
        const int lrow = lane >> 2, chunk = (lane & 3) ^ ((lrow >> 1) & 3);
        const int kleft = o.k - k0;
        const int rows = left < BM ? left : BM;
        const int bytes = kleft > 0 && rows > 0 ? ((rows - 1) * (int)o.ld + kleft) * 2 : 0;
        const __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc((void *)(base + k0), (short)0, bytes, 0x00020000);
        int off = chunk * 8 < kleft ? (row * (int)o.ld + chunk * 8) * 2 : 0x7FFFFFF0;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, LDS_ADDR(&lds[dst + kb * 1024]), 16, off, 0, 0, 0);
    };
    auto load_cols = [&](const TgOperand &o, int c0, int k0, int kb, int dst) __attribute__((always_inline)) {
        const int r = kb * (1024 / QRB) + lane / QCH, s16 = lane % QCH;
        const int kleft = o.k - k0, rows = kleft < kBK ? kleft : kBK;
        const int bytes = rows > 0 ? ((rows - 1) * (int)o.ld + (o.outer - c0)) * 2 : 0;
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            (void *)(o.p + (int64_t)k0 * o.ld + c0), (short)0, bytes, 0x00020000);
        const int col = (((s16 >> 1) ^ qsw(r)) << 4) + ((s16 & 1) << 3);
        int off = col < o.outer - c0 ? (r * (int)o.ld + col) * 2 : 0x7FFFFFF0;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, LDS_ADDR(&lds[dst + kb * 1024]), 16, off, 0, 0, 0);
    };

    for (int s = 0; s < P.nseg; ++s) {
        const TgSegment &S = P.seg[s];
        for (int st = 0; st < S.stages; ++st) {
            const int k0 = st * kBK;
            __syncthreads();
#pragma unroll
            for (int x = 0; x < LOADS; ++x) {
                const int kb = x * NW + wave;
                if constexpr (AKM) {
                    load_cols(S.a, m0, k0, kb, 0);
                } else {
                    load_rows(S.a, S.a.p + (int64_t)m0 * S.a.ld, S.a.outer - m0, k0, kb, kb * 16 + (lane >> 2), 0);
                }
                if constexpr (BKM) {
                    load_cols(S.b, n0, k0, kb, OPB);
                } else {
                    // LDS row n of block kb holds the tile's column
                    // 32 (kb / 2) + 8 (n / 4) + 4 (kb % 2) + n % 4; gate / up:
                    // block kb % 4 of wave kb / 4, gate in blocks 0, 1
                    const int n = lane >> 2;
                    const int sub = 8 * (n >> 2) + 4 * (kb & 1) + (n & 3);
                    const TgOperand &o = GLU && (kb & 2) ? P.seg[1].b : S.b;
                    const int row = (GLU ? (kb >> 2) * 32 : (kb >> 1) * 32) + sub;
                    load_rows(o, o.p + (int64_t)n0 * o.ld, o.outer - n0, k0, kb, row, OPB);
                }
            }
            __builtin_amdgcn_s_waitcnt(0);
            __syncthreads();
            bf16x8 fa[FM], fb[FN];
            const int fr = lane & 15, fh = lane >> 4;
            const int foff = fr * ROW + ((fh ^ ((fr >> 1) & 3)) << 4);
            const int tg = lane >> 4, tq = (lane >> 2) & 3, tp = lane & 3;
            const int tpo = ((tp >> 1) << 4) + ((tp & 1) << 3), tr = 8 * tg + tq;
            auto tread = [&](int unit, int op) __attribute__((always_inline)) {
                tg_u32x2 lo, hi;
                const uint32_t a = lds_base + op + tr * QRB + ((unit ^ qsw(tr)) << 5) + tpo;
                asm volatile("ds_read_b64_tr_b16 %0, %2\n\tds_read_b64_tr_b16 %1, %2 offset:%3\n\ts_waitcnt lgkmcnt(0)"
                             : "=&v"(lo), "=&v"(hi)
                             : "v"(a), "i"(4 * QRB)
                             : "memory");
                return __builtin_bit_cast(bf16x8, tg_u32x4{lo.x, lo.y, hi.x, hi.y});
            };
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                if constexpr (AKM)
                    fa[i] = tread(wr * (WTM / 16) + i, 0);
                else
                    fa[i] = *reinterpret_cast<const bf16x8 *>(&lds[wr * WTM * ROW + i * 16 * ROW + foff]);
            }
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                if constexpr (BKM)
                    fb[j] = tread(wc * (WTN / 16) + j, OPB);
                else
                    fb[j] = *reinterpret_cast<const bf16x8 *>(&lds[OPB + wc * WTN * ROW + j * 16 * ROW + foff]);
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
        }
        if (GLU) break;  // (the second segment holds the up projection's rows)
    }
    const int R0 = m0 + wr * WTM;
    if constexpr (EPI == kTgXent)
        xent_epilogue<FM>(L, acc, R0, n0 + wc * WTN, lane);
    else if constexpr (GLU)
        glu_epilogue<FM, EPI == kTgGluBack>(L, acc, R0, n0 + wc * 32, lane);
    else
        store_epilogue<FM, FN, !BKM>(L, P, acc, R0, n0 + wc * WTN, lane);
}

template <int BM, int EPI, bool AKM, bool BKM>
hipError_t run(TgLaunch &L, hipStream_t stream) {
    constexpr bool GLU = EPI == kTgGlu || EPI == kTgGluBack;
    constexpr int BN = GLU ? BM / 2 : BM;
    L.tiles_m = (L.M + BM - 1) / BM;
    L.tiles_n = (L.N + BN - 1) / BN;
    const int64_t grid = (int64_t)L.tiles_m * L.tiles_n * L.nprob;
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL((tg_kernel<BM, EPI, AKM, BKM>), dim3((uint32_t)grid), dim3(256), 0, stream, L);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_tg(TgEpilogue epi, bool a_km, bool b_km, TgLaunch &L, hipStream_t stream) {
    if (epi == kTgXent) return run<128, kTgXent, false, false>(L, stream);
    if (epi == kTgGlu) return run<128, kTgGlu, false, false>(L, stream);
    if (epi == kTgGluBack) return run<128, kTgGluBack, false, false>(L, stream);
    if (!b_km) return hipErrorInvalidValue;
    return a_km ? run<128, kTgStore, true, true>(L, stream) : run<128, kTgStore, false, true>(L, stream);
}

}  // namespace zopt
