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

// dst [rows, cp] = src [rows, cols], zero in [cols, cp) and in rows whose
// target is the ignored one (target != NULL); one thread an eight
__global__ __launch_bounds__(kThreads) void pad_copy_kernel(const uint16_t *__restrict__ src, int64_t ld,
                                                            int64_t rows, int64_t cols, int64_t cp,
                                                            uint16_t *__restrict__ dst,
                                                            const int64_t *__restrict__ target, int64_t ignore) {
    const int64_t per = cp / 8, total = rows * per;
    for (int64_t id = blockIdx.x * (int64_t)kThreads + threadIdx.x; id < total; id += (int64_t)gridDim.x * kThreads) {
        const int64_t r = id / per, c = (id - r * per) * 8;
        const int64_t left = cols - c;
        tg_u32x4 v{0, 0, 0, 0};
        if (target == nullptr || target[r] != ignore)
            v = tg_load8h(src + r * ld + c, left > 8 ? 8 : (int)left);
        *reinterpret_cast<tg_u32x4 *>(dst + r * cp + c) = v;
    }
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
// eight each.
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
        if (n > 0) p = tg_load8h(x + r * ld + c, n);
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

__global__ __launch_bounds__(kThreads) void act8_unpack_kernel(const uint8_t *__restrict__ q,
                                                               const uint8_t *__restrict__ scale, int64_t rows,
                                                               int64_t cols, uint16_t *__restrict__ x, int64_t ld,
                                                               int64_t cols_out) {
    const int64_t blocks = (cols + 31) / 32, per = (cols_out + 7) / 8, total = rows * per;
    for (int64_t id = blockIdx.x * (int64_t)kThreads + threadIdx.x; id < total; id += (int64_t)gridDim.x * kThreads) {
        const int64_t r = id / per, c = (id - r * per) * 8;
        const int64_t left = cols - c, lo = cols_out - c;
        const int n = left > 8 ? 8 : left < 0 ? 0 : (int)left;
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (n > 0) {
            tg_unpack_e4m3(tg_load8b(q + r * cols + c, n), tg_scale_out(scale[r * blocks + (c >> 5)]), v);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = k < n ? v[k] : 0.0f;
        }
        tg_store8h(x + r * ld + c, pack8(v), lo > 8 ? 8 : (int)lo);
    }
}

// The number of rows that take part, summed over a block of 1024 threads.
__device__ __forceinline__ long long valid_rows(const int64_t *__restrict__ target, int64_t rows, int64_t ignore) {
    __shared__ long long part[16];
    long long n = 0;
    for (int64_t i = threadIdx.x; i < rows; i += 1024) n += target[i] != ignore ? 1 : 0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = n;
    __syncthreads();
    long long all = 0;
    for (int k = 0; k < 16; ++k) all += part[k];
    return all;
}
__device__ __forceinline__ double share_of(long long rows, int mean) {
    return !mean ? 1.0 : rows > 0 ? 1.0 / (double)rows : 0.0;
}

// the gradients' factor
__global__ __launch_bounds__(1024) void xent_count_kernel(const int64_t *__restrict__ target, int64_t rows,
                                                          int64_t ignore, int mean, float grad_scale,
                                                          float *__restrict__ factor) {
    const long long n = mean ? valid_rows(target, rows, ignore) : 0;
    if (threadIdx.x == 0) *factor = (float)(share_of(n, mean) * (double)grad_scale);
}

// (m, s) of two sets of exponentials, s relative to exp(m)
__device__ __forceinline__ void join(float &m, float &s, float m2, float s2) {
    const float t = fmaxf(m, m2);
    const float ref = t == -INFINITY ? 0.0f : t;  // (a NaN maximum is left out here and makes the sum NaN)
    s = s * expf(m - ref) + s2 * expf(m2 - ref);
    m = t;
}

// lse = m + log(sum_g s_g exp(m_g - m)), m the largest group maximum.  A block
// of 1024 threads takes 16 rows, 64 threads a row; each joins every 64th
// group, eight at a time so that as many loads are in flight, and the 64 join
// in a fixed order.  A target outside [0, V) that is not the ignored one
// makes the row NaN.
__global__ __launch_bounds__(1024) void xent_lse_kernel(const float2 *__restrict__ stats, int64_t ldstat, int groups,
                                                        const int64_t *__restrict__ target, int64_t ignore, int V,
                                                        const float *__restrict__ zt, int64_t rows,
                                                        float *__restrict__ lse, float *__restrict__ row_loss) {
    __shared__ float pm[16][16], ps[16][16];
    const int lr = threadIdx.x & 15, part = threadIdx.x >> 4;
    const int64_t row = blockIdx.x * (int64_t)16 + lr;
    const bool live = row < rows;
    float m = -INFINITY, s = 0.0f;
    if (live) {
        const float2 *p = stats + row;
        for (int g = part; g < groups; g += 512) {
            float2 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = g + 64 * k < groups ? p[(int64_t)(g + 64 * k) * ldstat] : make_float2(-INFINITY, 0.0f);
            float t = m;
#pragma unroll
            for (int k = 0; k < 8; ++k) t = fmaxf(t, v[k].x);
            const float ref = t == -INFINITY ? 0.0f : t;
            s *= expf(m - ref);
#pragma unroll
            for (int k = 0; k < 8; ++k) s += v[k].y * expf(v[k].x - ref);
            m = t;
        }
    }
#pragma unroll
    for (int o = 16; o <= 32; o <<= 1) {
        const float m2 = __shfl_xor(m, o), s2 = __shfl_xor(s, o);
        join(m, s, m2, s2);
    }
    if ((part & 3) == 0) {
        pm[part >> 2][lr] = m;
        ps[part >> 2][lr] = s;
    }
    __syncthreads();
    if (part != 0 || !live) return;
    for (int k = 1; k < 16; ++k) join(m, s, pm[k][lr], ps[k][lr]);
    const int64_t t = target[row];
    const bool in = t >= 0 && t < V;
    const float ls = logf(s);
    lse[row] = in || t == ignore ? m + ls : NAN;
    row_loss[row] = t == ignore ? 0.0f : in ? ls + (m - zt[row]) : NAN;
}

// e -> P in place, eight columns a thread: exp(m_group - lse) e, 0 for ignored
// rows.  The target's own entry, softmax - 1, comes from the row's loss,
// expm1(-row_loss): where the model is sure of the target the difference is
// small, and e's 11 bits would be most of it.
__global__ __launch_bounds__(kThreads) void xent_probs_kernel(uint16_t *__restrict__ e, int64_t lde, int64_t rows,
                                                              int V, const float2 *__restrict__ stats, int64_t ldstat,
                                                              const float *__restrict__ lse,
                                                              const float *__restrict__ row_loss,
                                                              const int64_t *__restrict__ target, int64_t ignore) {
    const int64_t per = lde / 8, total = rows * per;
    for (int64_t id = blockIdx.x * (int64_t)kThreads + threadIdx.x; id < total; id += (int64_t)gridDim.x * kThreads) {
        const int64_t r = id / per, c = (id - r * per) * 8;
        tg_u32x4 *p = reinterpret_cast<tg_u32x4 *>(e + r * lde + c);
        const int64_t t = target[r];
        tg_u32x4 out{0, 0, 0, 0};
        if (t != ignore && c < V) {
            const tg_u32x4 in = *p;
            const float f = expf(stats[(c / kXentGroup) * ldstat + r].x - lse[r]);
            const int64_t rel = t - c;
            float v[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const tg_f16x2 h = __builtin_bit_cast(tg_f16x2, (uint32_t)in[k]);
                v[2 * k] = (float)h.x * f;
                v[2 * k + 1] = (float)h.y * f;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (rel == k) v[k] = expm1f(-row_loss[r]);
                if (c + k >= V) v[k] = 0.0f;
            }
            out = pack8(v);
        }
        *p = out;
    }
}

// loss = share * sum of row losses, in double, in a fixed order
__global__ __launch_bounds__(1024) void xent_total_kernel(const float *__restrict__ row_loss, int64_t rows,
                                                          const int64_t *__restrict__ target, int64_t ignore,
                                                          int mean, float *__restrict__ loss) {
    __shared__ double part[16];
    const long long n = mean ? valid_rows(target, rows, ignore) : 0;
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < rows; i += 1024) s += (double)row_loss[i];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0.0;
        for (int k = 0; k < 16; ++k) all += part[k];
        *loss = (float)(all * share_of(n, mean));
    }
}

// dg = dh u act'(g), du = dh act(g), h = act(g) u, eight columns a thread
__global__ __launch_bounds__(kThreads) void glu_back_act8_kernel(
    const uint8_t *__restrict__ g8, const uint8_t *__restrict__ gs, const uint8_t *__restrict__ u8,
    const uint8_t *__restrict__ us, const uint16_t *__restrict__ dh, int64_t lddh, int64_t rows, int64_t F, int act,
    uint16_t *__restrict__ dg, uint16_t *__restrict__ du, int64_t lddg, uint16_t *__restrict__ h, int64_t ldh) {
    const int64_t blocks = (F + 31) / 32, per = (F + 7) / 8, total = rows * per;
    for (int64_t id = blockIdx.x * (int64_t)kThreads + threadIdx.x; id < total; id += (int64_t)gridDim.x * kThreads) {
        const int64_t r = id / per, c = (id - r * per) * 8;
        const int n = F - c > 8 ? 8 : (int)(F - c);
        float g[8], u[8], d[8], og[8], ou[8], oh[8];
        tg_unpack_e4m3(tg_load8b(g8 + r * F + c, n), tg_scale_out(gs[r * blocks + (c >> 5)]), g);
        tg_unpack_e4m3(tg_load8b(u8 + r * F + c, n), tg_scale_out(us[r * blocks + (c >> 5)]), u);
        unpack8(tg_load8h(dh + r * lddh + c, n), d);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const TgActValue a = tg_act(g[k], act);
            og[k] = k < n ? d[k] * u[k] * a.da : 0.0f;
            ou[k] = k < n ? d[k] * a.a : 0.0f;
            oh[k] = a.a * u[k];
        }
        *reinterpret_cast<tg_u32x4 *>(dg + r * lddg + c) = pack8(og);
        *reinterpret_cast<tg_u32x4 *>(du + r * lddg + c) = pack8(ou);
        if (h != nullptr) tg_store8h(h + r * ldh + c, pack8(oh), n);
    }
}

}  // namespace

hipError_t launch_pad_copy(const uint16_t *src, int64_t ld, int64_t rows, int64_t cols, uint16_t *dst,
                           const int64_t *target, int64_t ignore, hipStream_t stream) {
    const int64_t cp = (cols + 7) / 8 * 8;
    hipLaunchKernelGGL(pad_copy_kernel, dim3(blocks_for(rows * (cp / 8))), dim3(kThreads), 0, stream, src, ld, rows,
                       cols, cp, dst, target, ignore);
    return hipGetLastError();
}

hipError_t launch_fill_zero(uint16_t *dst, int64_t ld, int64_t rows, int64_t cols, hipStream_t stream) {
    hipLaunchKernelGGL(fill_zero_kernel, dim3(blocks_for(rows * cols)), dim3(kThreads), 0, stream, dst, ld, rows, cols);
    return hipGetLastError();
}

hipError_t launch_act8_pack(const uint16_t *x, int64_t ld, int64_t rows, int64_t cols, uint8_t *q, uint8_t *scale,
                            hipStream_t stream) {
    hipLaunchKernelGGL(act8_pack_kernel, dim3(blocks_for(rows * ((cols + 31) / 32) * 4)), dim3(kThreads), 0, stream, x,
                       ld, rows, cols, q, scale);
    return hipGetLastError();
}

hipError_t launch_act8_unpack(const uint8_t *q, const uint8_t *scale, int64_t rows, int64_t cols, uint16_t *x,
                              int64_t ld, int64_t cols_out, hipStream_t stream) {
    hipLaunchKernelGGL(act8_unpack_kernel, dim3(blocks_for(rows * ((cols_out + 7) / 8))), dim3(kThreads), 0, stream, q,
                       scale, rows, cols, x, ld, cols_out);
    return hipGetLastError();
}

hipError_t launch_xent_count(const int64_t *target, int64_t rows, int64_t ignore, int32_t mean, float grad_scale,
                             float *factor, hipStream_t stream) {
    hipLaunchKernelGGL(xent_count_kernel, dim3(1), dim3(1024), 0, stream, target, rows, ignore, mean, grad_scale,
                       factor);
    return hipGetLastError();
}

hipError_t launch_xent_lse(const float2 *stats, int64_t ldstat, int32_t groups, const int64_t *target, int64_t ignore,
                           int32_t V, const float *zt, int64_t rows, float *lse, float *row_loss, hipStream_t stream) {
    hipLaunchKernelGGL(xent_lse_kernel, dim3((uint32_t)((rows + 15) / 16)), dim3(1024), 0, stream, stats, ldstat, groups,
                       target, ignore, V, zt, rows, lse, row_loss);
    return hipGetLastError();
}

hipError_t launch_xent_probs(uint16_t *e, int64_t lde, int64_t rows, int32_t V, const float2 *stats, int64_t ldstat,
                             const float *lse, const float *row_loss, const int64_t *target, int64_t ignore,
                             hipStream_t stream) {
    hipLaunchKernelGGL(xent_probs_kernel, dim3(blocks_for(rows * (lde / 8))), dim3(kThreads), 0, stream, e, lde, rows,
                       V, stats, ldstat, lse, row_loss, target, ignore);
    return hipGetLastError();
}

hipError_t launch_xent_total(const float *row_loss, int64_t rows, const int64_t *target, int64_t ignore, int32_t mean,
                             float *loss, hipStream_t stream) {
    hipLaunchKernelGGL(xent_total_kernel, dim3(1), dim3(1024), 0, stream, row_loss, rows, target, ignore, mean, loss);
    return hipGetLastError();
}

hipError_t launch_glu_back_act8(const uint8_t *g8, const uint8_t *gs, const uint8_t *u8, const uint8_t *us,
                                const uint16_t *dh, int64_t lddh, int64_t rows, int64_t F, int32_t act, uint16_t *dg,
                                uint16_t *du, int64_t lddg, uint16_t *h, int64_t ldh, hipStream_t stream) {
    hipLaunchKernelGGL(glu_back_act8_kernel, dim3(blocks_for(rows * ((F + 7) / 8))), dim3(kThreads), 0, stream, g8, gs,
                       u8, us, dh, lddh, rows, F, act, dg, du, lddg, h, ldh);
    return hipGetLastError();
}

}  // namespace zopt
