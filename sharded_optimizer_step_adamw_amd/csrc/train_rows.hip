// train_rows.hip -- the passes over rows around the matrix products of the
// gradient operators: padded copies, 8-bit checkpoints, the softmax's row
// statistics and probabilities, the gated block's pointwise backward.  All
// are bound by HBM.
#include "train_internal.h"

namespace zopt {
namespace {

constexpr int kThreads = 256;

// Blocks for n pieces of work, kThreads a block; the kernels stride over the
// rest.  2^20 blocks keep every index within the grid limits.
uint32_t blocks_for(int64_t n) {
    const int64_t b = (n + kThreads - 1) / kThreads;
    return (uint32_t)(b < 1 ? 1 : b > (1 << 20) ? (1 << 20) : b);
}

// The 16-bit side of an 8-bit checkpoint goes past the caches where it fills
// more than half of the memory-side one, and leaves that to the 8-bit side: a
// [8192, 14336] matrix packed and read back takes 120 us so, 139 us otherwise
// (a [8192, 4096] one 41 and 39).
bool past_half(int64_t bytes) { return bytes > kCacheBytes / 2; }

__device__ __forceinline__ void unpack8(tg_u32x4 p, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(p[k] << 16);
        v[2 * k + 1] = __uint_as_float(p[k] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ tg_u32x4 pack8(const float (&v)[8]) {
    return tg_u32x4{tg_pack_bf16(v[0], v[1]), tg_pack_bf16(v[2], v[3]), tg_pack_bf16(v[4], v[5]),
                    tg_pack_bf16(v[6], v[7])};
}

__global__ __launch_bounds__(kThreads) void fill_zero_kernel(uint16_t *__restrict__ dst, int64_t ld, int64_t rows,
                                                             int64_t cols) {
    const int64_t total = rows * cols;
    for (int64_t id = blockIdx.x * (int64_t)kThreads + threadIdx.x; id < total; id += (int64_t)gridDim.x * kThreads) {
        const int64_t r = id / cols;
        dst[r * ld + (id - r * cols)] = 0;
    }
}

// 8-bit checkpoints: four neighbouring threads hold a block of 32 values,
// eight each.  Bound by HBM: 5.2 to 5.5 TB/s on [8192, 14336] (64 to 69 us);
// reading back, with the 8-bit side still cached, 55 us.
template <bool PAST>
__global__ __launch_bounds__(kThreads) void act8_pack_kernel(const uint16_t *__restrict__ x, int64_t ld, int64_t rows,
                                                             int64_t cols, uint8_t *__restrict__ q,
                                                             uint8_t *__restrict__ scale) {
    const int64_t blocks = (cols + 31) / 32, total = rows * blocks * 4;
    // (total is a multiple of 4, so the four threads of a block stay together)
    for (int64_t id = blockIdx.x * (int64_t)kThreads + threadIdx.x; id < total; id += (int64_t)gridDim.x * kThreads) {
        const int64_t b = id >> 2, r = b / blocks, cb = b - r * blocks;
        const int64_t c = cb * 32 + (id & 3) * 8, left = cols - c;
        const int n = left > 8 ? 8 : left < 0 ? 0 : (int)left;
        tg_u32x4 p{0, 0, 0, 0};
        if (n > 0) p = tg_load8h<PAST>(x + r * ld + c, n);
        float v[8];
        unpack8(p, v);
        uint32_t big = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t a = __float_as_uint(v[k]) & 0x7FFFFFFFu;
            big = a > big ? a : big;
        }
        uint32_t o = __shfl_xor(big, 1);
        big = o > big ? o : big;
        o = __shfl_xor(big, 2);
        big = o > big ? o : big;
        const uint32_t byte = tg_scale_byte(big);
        if (n > 0) tg_store8b(q + r * cols + c, tg_pack_e4m3(v, byte), n);
        if ((id & 3) == 0) scale[b] = (uint8_t)byte;
    }
}

// eight values of row r from column c on
__device__ __forceinline__ void act8_values(const uint8_t *q, const uint8_t *scale, int64_t r, int64_t c, int64_t cols,
                                            int64_t blocks, int n, float (&v)[8]) {
    tg_unpack_e4m3(tg_load8b(q + r * cols + c, n), tg_scale_out(scale[r * blocks + (c >> 5)]), v);
}

template <bool PAST>
__global__ __launch_bounds__(kThreads) void act8_unpack_kernel(const uint8_t *__restrict__ q,
                                                               const uint8_t *__restrict__ scale, int64_t rows,
                                                               int64_t cols, uint16_t *__restrict__ x, int64_t ld) {
    const int64_t blocks = (cols + 31) / 32, per = (cols + 7) / 8, total = rows * per;
    for (int64_t id = blockIdx.x * (int64_t)kThreads + threadIdx.x; id < total; id += (int64_t)gridDim.x * kThreads) {
        const int64_t r = id / per, c = (id - r * per) * 8;
        const int n = cols - c > 8 ? 8 : (int)(cols - c);
        float v[8];
        act8_values(q, scale, r, c, cols, blocks, n, v);
        tg_store8h<PAST>(x + r * ld + c, pack8(v), n);
    }
}

// (m, s) of two sets of exponentials, s relative to exp(m)
__device__ __forceinline__ void join(float &m, float &s, float m2, float s2) {
    const float t = fmaxf(m, m2);
    const float ref = t == -INFINITY ? 0.0f : t;  // (a NaN maximum is left out here and makes the sum NaN)
    s = s * expf(m - ref) + s2 * expf(m2 - ref);
    m = t;
}

// One row a block: its loss from the group statistics,
//   lse = m + log(sum_g s_g exp(m_g - m)), m the largest group maximum,
//   row loss = lse - the target's logit,
// and, if e is wanted, its exponentials turned into P = softmax - onehot in
// place: exp(m_group - lse) e, 0 in columns [V, lde) and for ignored rows.
// Differences of logits come before anything is added to them, (m_group - m) -
// log sum, so that no error grows with the logits' size.
// The target's own entry, softmax - 1, comes from the row's loss,
// expm1(-row loss): where the model is sure of the target the difference is
// small, and e's 11 bits would be most of it; so it is off by the loss's
// error, about 2^-20, and like the loss has the right sign or is 0.  A target outside [0, V) that
// is not the ignored one makes the row NaN.  Everything is joined in a fixed
// order.  Bound by HBM: e is read and written once (4 bytes a logit), 5.1 TB/s
// on 8192 x 50304 (0.32 ms).
template <bool PAST>
__global__ __launch_bounds__(kThreads) void xent_rows_kernel(const float2 *__restrict__ stats, int groups,
                                                             const int64_t *__restrict__ target, int64_t ignore, int V,
                                                             const float *__restrict__ zt, int64_t rows,
                                                             float *__restrict__ row_loss, uint16_t *__restrict__ e,
                                                             int64_t lde) {
    __shared__ float pm[kThreads / 64], ps[kThreads / 64];
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const float2 *p = stats + row * groups;
        float m = -INFINITY, s = 0.0f;
        for (int g = threadIdx.x; g < groups; g += 4 * kThreads) {
            float2 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = g + k * kThreads < groups ? p[g + k * kThreads] : make_float2(-INFINITY, 0.0f);
            float t = m;
#pragma unroll
            for (int k = 0; k < 4; ++k) t = fmaxf(t, v[k].x);
            const float ref = t == -INFINITY ? 0.0f : t;  // (a NaN maximum is left out and makes the sum NaN)
            s *= expf(m - ref);
#pragma unroll
            for (int k = 0; k < 4; ++k) s += v[k].y * expf(v[k].x - ref);
            m = t;
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const float m2 = __shfl_xor(m, o), s2 = __shfl_xor(s, o);
            join(m, s, m2, s2);
        }
        __syncthreads();  // (the last row's values have been read)
        if ((threadIdx.x & 63) == 0) {
            pm[threadIdx.x >> 6] = m;
            ps[threadIdx.x >> 6] = s;
        }
        __syncthreads();
        m = pm[0];
        s = ps[0];
#pragma unroll
        for (int k = 1; k < kThreads / 64; ++k) join(m, s, pm[k], ps[k]);
        const int64_t t = target[row];
        const bool in = t >= 0 && t < V, used = t != ignore;
        const float ls = in ? logf(s) : NAN;
        const float loss = !used ? 0.0f : in ? ls + (m - zt[row]) : NAN;
        if (threadIdx.x == 0) row_loss[row] = loss;
        if (e == nullptr) continue;
        for (int64_t c = threadIdx.x * 8; c < lde; c += kThreads * 8) {
            tg_u32x4 *at = reinterpret_cast<tg_u32x4 *>(e + row * lde + c);
            tg_u32x4 out{0, 0, 0, 0};
            if (used && c < V) {
                const tg_u32x4 raw = tg_load<tg_u32x4, PAST>(at);
                const float f = expf((p[c / kXentGroup].x - m) - ls);
                const int64_t rel = t - c;
                float v[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const tg_f16x2 h = __builtin_bit_cast(tg_f16x2, (uint32_t)raw[k]);
                    v[2 * k] = (float)h.x * f;
                    v[2 * k + 1] = (float)h.y * f;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (rel == k) v[k] = expm1f(-loss);
                    if (c + k >= V) v[k] = 0.0f;
                }
                out = pack8(v);
            }
            tg_store<PAST>(at, out);
        }
    }
}

// loss = share * sum of row losses, in double, in a fixed order
__global__ __launch_bounds__(1024) void xent_total_kernel(TgTotal t) { tg_total<1024>(t); }

// The jobs before a call's products, each on blocks of its own; eight columns
// a thread.  One launch for all: each of them alone takes 3 to 5 us on small
// operands, most of it a launch's.
__device__ __forceinline__ void prep_copy(const TgPrep &j, int64_t block) {
    const int64_t per = (j.cols + 7) / 8, total = j.rows * per;
    for (int64_t id = block * kThreads + threadIdx.x; id < total; id += (int64_t)j.blocks * kThreads) {
        const int64_t r = id / per, c = (id - r * per) * 8, left = j.cols - c;
        tg_u32x4 v{0, 0, 0, 0};
        if (j.target == nullptr || j.target[r] != j.ignore)
            v = tg_load8h(j.src + r * j.ld + c, left > 8 ? 8 : (int)left);
        *reinterpret_cast<tg_u32x4 *>(j.dst + id * 8) = v;
    }
}
__device__ __forceinline__ void prep_unpack(const TgPrep &j, int64_t block) {
    const int64_t blocks = (j.cols + 31) / 32, per = (j.cols + 7) / 8, total = j.rows * per;
    for (int64_t id = block * kThreads + threadIdx.x; id < total; id += (int64_t)j.blocks * kThreads) {
        const int64_t r = id / per, c = (id - r * per) * 8;
        const int n = j.cols - c > 8 ? 8 : (int)(j.cols - c);
        float v[8];
        act8_values(j.q, j.scale, r, c, j.cols, blocks, n, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < n ? v[k] : 0.0f;
        *reinterpret_cast<tg_u32x4 *>(j.dst + id * 8) = pack8(v);
    }
}
// dg = dh u act'(g), du = dh act(g), h = act(g) u
__device__ __forceinline__ void prep_back(const TgPrep &j, int64_t block) {
    const int64_t blocks = (j.cols + 31) / 32, per = (j.cols + 7) / 8, total = j.rows * per;
    for (int64_t id = block * kThreads + threadIdx.x; id < total; id += (int64_t)j.blocks * kThreads) {
        const int64_t r = id / per, c = (id - r * per) * 8;
        const int n = j.cols - c > 8 ? 8 : (int)(j.cols - c);
        float g[8], u[8], d[8], og[8], ou[8], oh[8];
        act8_values(j.q, j.scale, r, c, j.cols, blocks, n, g);
        act8_values(j.q2, j.scale2, r, c, j.cols, blocks, n, u);
        unpack8(tg_load8h(j.src + r * j.ld + c, n), d);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const TgActValue a = tg_act(g[k], j.act);
            og[k] = k < n ? d[k] * u[k] * a.da : 0.0f;
            ou[k] = k < n ? d[k] * a.a : 0.0f;
            oh[k] = a.a * u[k];
        }
        *reinterpret_cast<tg_u32x4 *>(j.dst + r * j.dst_ld + c) = pack8(og);
        *reinterpret_cast<tg_u32x4 *>(j.dst2 + r * j.dst_ld + c) = pack8(ou);
        if (j.h != nullptr) tg_store8h(j.h + r * j.h_ld + c, pack8(oh), n);
    }
}
__device__ __forceinline__ void prep_count(const TgPrep &j) {
    const long long n = j.mean ? tg_valid_rows<kThreads>(j.target, j.rows, j.ignore) : 0;
    if (threadIdx.x == 0) *j.factor = (float)(tg_share(n, j.mean) * (double)j.grad_scale);
}
__global__ __launch_bounds__(kThreads) void prep_kernel(TgPrepList list) {
    uint32_t block = blockIdx.x;
    int k = 0;
    while (k + 1 < list.n && block >= list.job[k].blocks) block -= list.job[k++].blocks;
    const TgPrep &j = list.job[k];
    if (j.kind == kPrepCopy)
        prep_copy(j, block);
    else if (j.kind == kPrepUnpack)
        prep_unpack(j, block);
    else if (j.kind == kPrepBack)
        prep_back(j, block);
    else
        prep_count(j);
}

}  // namespace

hipError_t launch_prep(TgPrepList &list, hipStream_t stream) {
    if (list.n == 0) return hipSuccess;
    uint32_t total = 0;
    for (int k = 0; k < list.n; ++k) {
        TgPrep &j = list.job[k];
        j.blocks = j.kind == kPrepCount ? 1 : blocks_for(j.rows * ((j.cols + 7) / 8));
        total += j.blocks;
    }
    hipLaunchKernelGGL(prep_kernel, dim3(total), dim3(kThreads), 0, stream, list);
    return hipGetLastError();
}

hipError_t launch_fill_zero(uint16_t *dst, int64_t ld, int64_t rows, int64_t cols, hipStream_t stream) {
    hipLaunchKernelGGL(fill_zero_kernel, dim3(blocks_for(rows * cols)), dim3(kThreads), 0, stream, dst, ld, rows, cols);
    return hipGetLastError();
}

hipError_t launch_act8_pack(const uint16_t *x, int64_t ld, int64_t rows, int64_t cols, uint8_t *q, uint8_t *scale,
                            hipStream_t stream) {
    const auto kernel = past_half(rows * cols * 2) ? act8_pack_kernel<true> : act8_pack_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3(blocks_for(rows * ((cols + 31) / 32) * 4)), dim3(kThreads), 0, stream, x, ld, rows,
                       cols, q, scale);
    return hipGetLastError();
}

hipError_t launch_act8_unpack(const uint8_t *q, const uint8_t *scale, int64_t rows, int64_t cols, uint16_t *x,
                              int64_t ld, hipStream_t stream) {
    const auto kernel = past_half(rows * cols * 2) ? act8_unpack_kernel<true> : act8_unpack_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3(blocks_for(rows * ((cols + 7) / 8))), dim3(kThreads), 0, stream, q, scale, rows,
                       cols, x, ld);
    return hipGetLastError();
}

hipError_t launch_xent_rows(const float2 *stats, int32_t groups, const int64_t *target, int64_t ignore, int32_t V,
                            const float *zt, int64_t rows, float *row_loss, uint16_t *e, int64_t lde, bool past,
                            hipStream_t stream) {
    const auto kernel = past ? xent_rows_kernel<true> : xent_rows_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(rows < (1 << 20) ? rows : 1 << 20)), dim3(kThreads), 0, stream, stats,
                       groups, target, ignore, V, zt, rows, row_loss, e, lde);
    return hipGetLastError();
}

hipError_t launch_xent_total(const TgTotal &t, hipStream_t stream) {
    hipLaunchKernelGGL(xent_total_kernel, dim3(1), dim3(1024), 0, stream, t);
    return hipGetLastError();
}

}  // namespace zopt
