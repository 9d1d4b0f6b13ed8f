// rope.hip -- norms of queries and keys for each head with the rotation to
// their positions, and their gradients.
#include <cmath>

#include "lanes.h"
#include "rope_internal.h"

namespace zopt {
namespace {

constexpr int kThreads = 256;

// V 16-bit values as they lie in memory
template <int V>
struct Raw {
    uint32_t v[V > 1 ? V / 2 : 1];
};
template <int V, bool PAST>
__device__ __forceinline__ Raw<V> load_raw(const uint16_t *p) {
    Raw<V> r;
    if constexpr (V == 8) {
        const tg_u32x4 x = tg_load<tg_u32x4, PAST>(p);
#pragma unroll
        for (int k = 0; k < 4; ++k) r.v[k] = x[k];
    } else if constexpr (V == 4) {
        const tg_u32x2 x = tg_load<tg_u32x2, PAST>(p);
        r.v[0] = x.x;
        r.v[1] = x.y;
    } else if constexpr (V == 2) {
        r.v[0] = tg_load<uint32_t>(p);
    } else {
        r.v[0] = p[0];
    }
    return r;
}
template <int V>
__device__ __forceinline__ void widen(const Raw<V> &r, float *v) {
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = __uint_as_float(k & 1 ? r.v[k / 2] & 0xFFFF0000u : r.v[k / 2] << 16);
}
template <int V, bool PAST>
__device__ __forceinline__ void store_part(uint16_t *p, const float *v) {
    if constexpr (V == 8) {
        tg_store<PAST>(p, tg_u32x4{tg_pack_bf16(v[0], v[1]), tg_pack_bf16(v[2], v[3]), tg_pack_bf16(v[4], v[5]),
                             tg_pack_bf16(v[6], v[7])});
    } else if constexpr (V == 4) {
        tg_store<PAST>(p, tg_u32x2{tg_pack_bf16(v[0], v[1]), tg_pack_bf16(v[2], v[3])});
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) p[k] = (uint16_t)tg_pack_bf16(v[k], 0.0f);
    }
}

// Pairs turned by the angles of (cosine, sine) cs, by their negatives if BACK
template <int V, bool BACK>
__device__ __forceinline__ void turn(float (&v)[2 * V], const float2 (&cs)[V], int pairs) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const float c = cs[k].x, s = BACK ? -cs[k].y : cs[k].y;
        if (pairs) {
            const float a = v[2 * k], b = v[2 * k + 1];
            v[2 * k] = a * c - b * s;
            v[2 * k + 1] = b * c + a * s;
        } else {
            const float a = v[k], b = v[V + k];
            v[k] = a * c - b * s;
            v[V + k] = b * c + a * s;
        }
    }
}

// A row (one head of one token) is held by `group` lanes: a lane has NP pieces
// of 2 V elements, V of them where the first of each turned pair lies, V where
// the second does (style pairs, and elements that do not turn: 2 V neighbours),
// so that a rotation needs no other lane, and a row's two sums (of squares, and
// back of g n w) are joined in registers.  A block walks rows of one side, the
// next row's elements on their way while it works on one.
// Bound by HBM in pieces of 16 bytes (V = 8): 65536 tokens of 32 + 8 heads of 128 take
// 240 us forward (1.34 GB, 5.6 TB/s; a 2 GiB copy reaches 4.97) and 363 back (2.01 GB, 5.55);
// 8-byte pieces on twice the lanes took 297 and 396.  Smaller pieces, which a width or a
// turned part that is no multiple of 2 V leaves, are bound by instruction issue, and most
// where lanes of a row have nothing: heads of 96 with 24 turned (V = 4, 1.01 GB forward) 284
// and 359 us, of 80 with 20 (V = 2, 0.84 GB) 474 and 629, of 128 with 62 (V = 1) 975 and 1496,
// of 66 (V = 1, 33 of a wave's lanes, 0.69 GB) 939 and 1476.
// What only rows of a kind need (no position, one past the table, squares past fp32's
// range) is done in the waves that have one.
template <int V, int NP, bool BACK, bool PAST>
__global__ __launch_bounds__(kThreads, 4) void rope_kernel(RopeArgs a) {
    const bool second = (int)blockIdx.x >= a.first_blocks;
    const RopeSide &S = a.side[second ? 1 : 0];
    const int block = second ? blockIdx.x - a.first_blocks : blockIdx.x;
    const int blocks = second ? a.blocks - a.first_blocks : a.first_blocks;
    const int lane = threadIdx.x & 63, G = a.group, gl = lane & (G - 1), per = kThreads / G;
    const int half = a.rot / 2, turned = a.rot / (2 * V), pieces = (a.width + 2 * V - 1) / (2 * V);
    int at[NP], at2[NP];
    bool have[NP], have2[NP], turns[NP];
    float w[NP][2 * V], dw[NP][2 * V];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        const int p = gl + j * G;
        have[j] = p < pieces;
        turns[j] = p < turned;
        at[j] = turns[j] && !a.pairs ? V * p : 2 * V * p;
        at2[j] = turns[j] && !a.pairs ? half + V * p : 2 * V * p + V;
        have2[j] = have[j] && at2[j] < a.width;
#pragma unroll
        for (int k = 0; k < 2 * V; ++k) {
            w[j][k] = 1.0f;
            dw[j][k] = 0.0f;
        }
        if (S.w != nullptr) {
            if (have[j]) widen<V>(load_raw<V, false>(S.w + at[j]), &w[j][0]);
            if (have2[j]) widen<V>(load_raw<V, false>(S.w + at2[j]), &w[j][V]);
        }
    }
    const float inv_width = 1.0f / (float)a.width;
    const int64_t rows = a.tokens * S.heads, step = (int64_t)blocks * per;
    int64_t row = (int64_t)block * per + threadIdx.x / G;
    int64_t t = row / S.heads;
    int head = (int)(row - t * S.heads);
    const int64_t step_t = step / S.heads;
    const int step_h = (int)(step - step_t * S.heads);
    // A row's position and elements, read a row ahead of their use
    struct Row {
        int64_t pos;
        Raw<V> x[NP], x2[NP], d[NP], d2[NP];
    };
    auto fetch = [&](Row &R) __attribute__((always_inline)) {
        R.pos = -1;
        if (row < rows) R.pos = a.position != nullptr ? a.position[t] : t;
        if (row >= rows) return;
        const uint16_t *p = S.x + t * S.xt + head * S.xh, *q = S.dy + t * S.dt + head * S.dh;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            if (have[j]) R.x[j] = load_raw<V, PAST>(p + at[j]);
            if (have2[j]) R.x2[j] = load_raw<V, PAST>(p + at2[j]);
            if constexpr (BACK) {
                if (have[j]) R.d[j] = load_raw<V, PAST>(q + at[j]);
                if (have2[j]) R.d2[j] = load_raw<V, PAST>(q + at2[j]);
            }
        }
    };
    auto advance = [&]() __attribute__((always_inline)) {
        row += step;
        t += step_t;
        head += step_h;
        if (head >= S.heads) {
            head -= S.heads;
            ++t;
        }
    };
    Row cur, next;
    fetch(cur);
    // (all lanes of a wave stay in the loop: the sums below are over lanes)
    for (int64_t base = row - threadIdx.x / G; base < rows; base += step) {
        const bool live = row < rows;
        uint16_t *const out = S.out + t * S.ot + head * S.oh;
        const int64_t pos = cur.pos;
        const bool none = pos < 0, known = !none && pos < a.positions;
        const bool strange = __ballot(!known) != 0;
        float x[NP][2 * V], d[NP][2 * V];
        float2 cs[NP][V];
#pragma unroll
        for (int j = 0; j < NP; ++j) {
#pragma unroll
            for (int k = 0; k < V; ++k) cs[j][k] = make_float2(1.0f, 0.0f);
            if (known && turns[j]) __builtin_memcpy(cs[j], a.table + pos * half + V * (gl + j * G), sizeof(float2) * V);
        }
        advance();
        fetch(next);
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            widen<V>(cur.x[j], &x[j][0]);
            widen<V>(cur.x2[j], &x[j][V]);
            if constexpr (BACK) {
                widen<V>(cur.d[j], &d[j][0]);
                widen<V>(cur.d2[j], &d[j][V]);
            }
            // (places past the row's end add nothing)
#pragma unroll
            for (int k = 0; k < 2 * V; ++k) {
                const bool in = k < V ? have[j] : have2[j];
                x[j][k] = in ? x[j][k] : 0.0f;
                if constexpr (BACK) d[j][k] = in ? d[j][k] : 0.0f;
            }
        }
        if (__builtin_expect(strange, 0)) {
            // (a row without a position is zeros, one whose position the table lacks is NaN)
#pragma unroll
            for (int j = 0; j < NP; ++j)
#pragma unroll
                for (int k = 0; k < 2 * V; ++k) {
                    const float fill = none || !(k < V ? have[j] : have2[j]) ? 0.0f : NAN;
                    x[j][k] = known ? x[j][k] : fill;
                    if constexpr (BACK) d[j][k] = known ? d[j][k] : fill;
                }
        }
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int k = 0; k < 2 * V; ++k) ss += x[j][k] * x[j][k];
        cur = next;
        ss = group_sum(ss, G);
        // A row whose squares pass fp32's range, or lie so far down that some that count are
        // no normal numbers (which needs an eps of next to nothing), is multiplied by a
        // power of two first: r is 0 or above 2^40 then, of rows without a position too.
        float r = 1.0f / sqrtf(ss * inv_width + a.eps);
        const bool odd = __float_as_uint(r) - 1 >= __float_as_uint(0x1p40f), rescaled = __ballot(odd) != 0;
        const float factor = !odd ? 1.0f : r == 0.0f ? 0x1p-70f : 0x1p70f;
        if (__builtin_expect(rescaled, 0)) {
            float sq = 0.0f;
#pragma unroll
            for (int j = 0; j < NP; ++j)
#pragma unroll
                for (int k = 0; k < 2 * V; ++k) {
                    x[j][k] *= factor;
                    sq += x[j][k] * x[j][k];
                }
            sq = group_sum(sq, G);
            r = 1.0f / sqrtf(sq * inv_width + a.eps * factor * factor);
        }
        r = none ? 0.0f : r;
        if constexpr (!BACK) {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
#pragma unroll
                for (int k = 0; k < 2 * V; ++k) x[j][k] = x[j][k] * r * w[j][k];
                if (turns[j]) turn<V, false>(x[j], cs[j], a.pairs);
            }
        } else {
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                if (turns[j]) turn<V, true>(d[j], cs[j], a.pairs);
#pragma unroll
                for (int k = 0; k < 2 * V; ++k) {
                    x[j][k] *= r;
                    dw[j][k] += d[j][k] * x[j][k];
                    d[j][k] *= w[j][k];
                    m += d[j][k] * x[j][k];
                }
            }
            m = group_sum(m, G) * inv_width;
#pragma unroll
            for (int j = 0; j < NP; ++j)
#pragma unroll
                for (int k = 0; k < 2 * V; ++k) x[j][k] = r * (d[j][k] - x[j][k] * m);
            if (__builtin_expect(rescaled, 0)) {
#pragma unroll
                for (int j = 0; j < NP; ++j)
#pragma unroll
                    for (int k = 0; k < 2 * V; ++k) x[j][k] *= factor;
            }
        }
        if (__builtin_expect(strange, 0)) {  // (zeros whatever the weights are)
#pragma unroll
            for (int j = 0; j < NP; ++j)
#pragma unroll
                for (int k = 0; k < 2 * V; ++k) x[j][k] = none ? 0.0f : x[j][k];
        }
        if (live) {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                if (have[j]) store_part<V, PAST>(out + at[j], &x[j][0]);
                if (have2[j]) store_part<V, PAST>(out + at2[j], &x[j][V]);
            }
        }
    }
    if constexpr (BACK) {
        if (S.dw == nullptr) return;
        // the block's sums: over the rows of a wave, then over the waves, in order
        extern __shared__ float sums[];  // [waves][width]
        const int wave = threadIdx.x >> 6;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
#pragma unroll
            for (int k = 0; k < 2 * V; ++k) {
                float v = dw[j][k];
                for (int o = G; o < 64; o <<= 1) v += __shfl_xor(v, o);
                const int e = k < V ? at[j] + k : at2[j] + k - V;
                if (lane < G && (k < V ? have[j] : have2[j])) sums[wave * a.width + e] = v;
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < a.width; e += kThreads) {
            float v = sums[e];
#pragma unroll
            for (int k = 1; k < kThreads / 64; ++k) v += sums[k * a.width + e];
            a.part[(int64_t)blockIdx.x * a.width + e] = v;
        }
    }
}

// dw from the blocks' sums: a block 16 columns of one side, 64 threads each,
// which add every 64th block's, then those in order.
__global__ __launch_bounds__(1024) void rope_dw_kernel(RopeArgs a) {
    __shared__ float sums[64][17];
    const int each = (a.width + 15) / 16, side = blockIdx.x / each, c = threadIdx.x & 15, r = threadIdx.x >> 4;
    const int e = (blockIdx.x - side * each) * 16 + c;
    const RopeSide &S = a.side[side];
    const int b0 = side == 0 ? 0 : a.first_blocks, b1 = side == 0 ? a.first_blocks : a.blocks;
    float v = 0.0f;
    if (e < a.width) {
#pragma unroll 8
        for (int b = b0 + r; b < b1; b += 64) v += a.part[(int64_t)b * a.width + e];
    }
    sums[r][c] = v;
    __syncthreads();
    if (r == 0 && e < a.width && S.dw != nullptr) {
        v = 0.0f;
#pragma unroll 8
        for (int k = 0; k < 64; ++k) v += sums[k][c];
        S.dw[e] = (uint16_t)tg_pack_bf16(v, 0.0f);
    }
}

// The angle of pair i at position p is p base^(-2 i / rot): in 64 bits, since
// far positions' angles have few bits left behind the point in 32.
__global__ __launch_bounds__(kThreads) void rope_table_kernel(int64_t positions, int half, double base,
                                                              float2 *__restrict__ table) {
    const int64_t total = positions * half;
    for (int64_t id = blockIdx.x * (int64_t)kThreads + threadIdx.x; id < total; id += (int64_t)gridDim.x * kThreads) {
        const int64_t p = id / half;
        const int i = (int)(id - p * half);
        double s, c;
        sincos((double)p * pow(base, -(double)i / (double)half), &s, &c);
        table[id] = make_float2((float)c, (float)s);
    }
}

// The widest piece that divides the row and its turned part.
int piece(const RopeArgs &a) {
    for (int v : {8, 4, 2})
        if (a.width % (2 * v) == 0 && a.rot % (2 * v) == 0) return v;
    return 1;
}
template <bool BACK, bool PAST>
hipError_t run(const RopeArgs &a, hipStream_t stream) {
    const size_t lds = BACK ? (size_t)(kThreads / 64) * a.width * 4 : 0;
    const dim3 grid((uint32_t)a.blocks), block(kThreads);
    switch (piece(a)) {
        case 8: hipLaunchKernelGGL((rope_kernel<8, 1, BACK, PAST>), grid, block, lds, stream, a); break;
        case 4: hipLaunchKernelGGL((rope_kernel<4, 1, BACK, PAST>), grid, block, lds, stream, a); break;
        case 2: hipLaunchKernelGGL((rope_kernel<2, 2, BACK, PAST>), grid, block, lds, stream, a); break;
        default: hipLaunchKernelGGL((rope_kernel<1, 4, BACK, PAST>), grid, block, lds, stream, a); break;
    }
    return hipGetLastError();
}
template <bool BACK>
hipError_t run(const RopeArgs &a, hipStream_t stream) {
    // Rows that do not fit the memory-side cache go past it: 65536 tokens of 40
    // heads of 128 take 240 us forward and 363 back so, 256 and 409 otherwise; 8192
    // (84 MB in) the same either way.
    const int64_t bytes = a.tokens * (a.side[0].heads + a.side[1].heads) * a.width * 2 * (BACK ? 3 : 2);
    return bytes > 2 * kCacheBytes ? run<BACK, true>(a, stream) : run<BACK, false>(a, stream);
}

}  // namespace

void plan_rope(RopeArgs &a) {
    const int v = piece(a), pieces = (a.width + 2 * v - 1) / (2 * v);
    int g = 1;
    while (g < pieces && g < 64) g <<= 1;
    a.group = g;
    // (as many blocks as the GPU's 256 CUs hold: the call above takes 240 us forward with
    // 1024, 251 with 4096; backward, whose blocks' sums are added up, 363, 367 with 2048 and 372
    // with 4096)
    const int64_t per = kThreads / g, most = 1024;
    const int64_t q = (a.tokens * a.side[0].heads + per - 1) / per, k = (a.tokens * a.side[1].heads + per - 1) / per;
    int64_t bq = q, bk = k;
    if (q + k > most) {
        bq = most * q / (q + k);
        if (bq < 1) bq = 1;
        if (bq >= most && k > 0) bq = most - 1;
        bk = k > 0 ? most - bq : 0;
    }
    a.first_blocks = (int32_t)bq;
    a.blocks = (int32_t)(bq + bk);
}

hipError_t launch_rope(const RopeArgs &a, hipStream_t stream) { return run<false>(a, stream); }

hipError_t launch_rope_back(const RopeArgs &a, hipStream_t stream) {
    hipError_t e = a.blocks > 0 ? run<true>(a, stream) : hipSuccess;
    if (e == hipSuccess && (a.side[0].dw != nullptr || a.side[1].dw != nullptr)) {
        hipLaunchKernelGGL(rope_dw_kernel, dim3((uint32_t)((a.width + 15) / 16 * 2)), dim3(1024), 0, stream, a);
        e = hipGetLastError();
    }
    return e;
}

hipError_t launch_rope_table(int64_t positions, int32_t rot, double base, float2 *table, hipStream_t stream) {
    const int64_t n = positions * (rot / 2), b = (n + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(rope_table_kernel, dim3((uint32_t)(b < (1 << 20) ? b : 1 << 20)), dim3(kThreads), 0, stream,
                       positions, rot / 2, base, table);
    return hipGetLastError();
}

}  // namespace zopt
