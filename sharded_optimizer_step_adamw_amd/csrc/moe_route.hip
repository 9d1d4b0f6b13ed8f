// moe_route.hip -- routing of tokens to experts: scores, choice, weights, the
// slots' order by expert, and the logits' gradient.
#include <cmath>

#include "moe_internal.h"

namespace zopt {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

__device__ __forceinline__ float read_logit(const void *p, int64_t i, bool bf16) {
    return bf16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p)[i] << 16)
                : reinterpret_cast<const float *>(p)[i];
}

// max / sum over the G lanes of a token
__device__ __forceinline__ float group_max(float v, int G) {
    for (int o = 1; o < G; o <<= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ float group_sum(float v, int G) {
    for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o);
    return v;
}

// log of the logistic function
__device__ __forceinline__ float log_logistic(float z) { return fminf(z, 0.0f) - log1pf(expf(-fabsf(z))); }
__device__ __forceinline__ float logistic(float z) {
    const float e = expf(-fabsf(z));
    return (z >= 0.0f ? 1.0f : e) / (1.0f + e);
}

// G lanes a token, NV experts a lane (expert lane + G i).
template <int NV>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a, int G) {
    extern __shared__ double lds[];
    const int E = a.experts;
    int *hist = reinterpret_cast<int *>(lds);
    double *keys = lds + (E + 1) / 2;
    const int lane = threadIdx.x & 63, gl = lane & (G - 1), first_lane = lane - gl;
    const int per = kThreads / G, own = threadIdx.x / G;
    const bool scored = a.bias != nullptr || a.groups > 1;
    double *row_keys = keys + (int64_t)own * (E + a.groups), *row_groups = row_keys + E;
    for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * a.block_tokens;
    const int64_t t1 = t0 + a.block_tokens < a.tokens ? t0 + a.block_tokens : a.tokens;
    for (int64_t base = t0; base < t1; base += per) {
        const int64_t t = base + own;
        const bool live = t < t1;
        float z[NV];
        double key[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = gl + G * i;
            z[i] = live && e < E ? read_logit(a.logits, t * a.ld + e, a.bf16) : -INFINITY;
        }
        float top = -INFINITY, sum = 0.0f;
        if (!a.sigmoid) {
#pragma unroll
            for (int i = 0; i < NV; ++i) top = fmaxf(top, z[i]);
            top = group_max(top, G);
            const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int i = 0; i < NV; ++i) sum += z[i] == -INFINITY ? 0.0f : expf(z[i] - ref);
            sum = group_sum(sum, G);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = (double)z[i];
        if (scored) {
            double total = 0.0;
            if (!a.sigmoid) {
                const double ref = top == -INFINITY ? 0.0 : (double)top;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    key[i] = z[i] == -INFINITY ? 0.0 : exp((double)z[i] - ref);
                    total += key[i];
                }
                for (int o = 1; o < G; o <<= 1) total += __shfl_xor(total, o);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = gl + G * i;
                double p = a.sigmoid ? 1.0 / (1.0 + exp(-(double)z[i])) : key[i] / total;
                if (a.bias != nullptr && e < E) p += (double)a.bias[e];
                key[i] = z[i] == -INFINITY ? -INFINITY : p;
            }
        }
        // a NaN ranks behind every number
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = key[i] != key[i] ? -1.7976931348623157e308 : key[i];
        if (a.groups > 1) {
            const int size = E / a.groups;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (gl + G * i < E) row_keys[gl + G * i] = key[i];
            __syncthreads();
            for (int g = gl; g < a.groups; g += G) {
                double b1 = -INFINITY, b2 = -INFINITY;
                for (int i = 0; i < size; ++i) {
                    const double k = row_keys[g * size + i];
                    if (k > b1) {
                        b2 = b1;
                        b1 = k;
                    } else if (k > b2) {
                        b2 = k;
                    }
                }
                row_groups[g] = b2 == -INFINITY ? b1 : b1 + b2;
            }
            __syncthreads();
            // an expert stays if fewer than top_groups groups come before its own
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = gl + G * i;
                if (e >= E) continue;
                const int g = e / size;
                const double own_key = row_groups[g];
                int before = 0;
                for (int h = 0; h < a.groups; ++h)
                    before += row_groups[h] > own_key || (row_groups[h] == own_key && h < g) ? 1 : 0;
                if (before >= a.top_groups) key[i] = -INFINITY;
            }
            __syncthreads();
        }
        // the best k, one after the other; lane j keeps the j-th
        int chosen = -1;
        float zc = -INFINITY;
        for (int j = 0; j < a.top; ++j) {
            double best = -INFINITY;
            int at = 0x7FFFFFFF;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at = gl + G * i;
                }
            for (int o = 1; o < G; o <<= 1) {
                const double b = __shfl_xor(best, o);
                const int n = __shfl_xor(at, o);
                if (b > best || (b == best && n < at)) {
                    best = b;
                    at = n;
                }
            }
            const bool some = best > -INFINITY;
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (gl + G * i == at) {
                    v = z[i];
                    key[i] = -INFINITY;
                }
            v = __shfl(v, first_lane + (some ? at & (G - 1) : 0));
            if (gl == j) {
                chosen = some ? at : -1;
                zc = v;
            }
        }
        float w = 0.0f;
        if (a.renormalise) {
            const float l = chosen < 0 ? -INFINITY : a.sigmoid ? log_logistic(zc) : zc;
            const float m = group_max(l, G);
            const float e = chosen < 0 ? 0.0f : expf(l - m);
            const float s = group_sum(e, G);
            w = chosen < 0 ? 0.0f : a.scale * (e / s);
        } else if (chosen >= 0) {
            w = a.scale * (a.sigmoid ? logistic(zc) : expf(zc - top) / sum);
        }
        if (live && gl < a.top) {
            a.chosen[t * a.top + gl] = chosen;
            a.weights[t * a.top + gl] = w;
            if (chosen >= 0) atomicAdd(&hist[chosen], 1);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) a.counts[(int64_t)blockIdx.x * E + e] = hist[e];
}

__global__ __launch_bounds__(kThreads) void plan_count_kernel(PlanArgs a) {
    extern __shared__ int hist[];
    for (int e = threadIdx.x; e < a.experts; e += kThreads) hist[e] = 0;
    __syncthreads();
    const int64_t each = (int64_t)a.block_tokens * a.top, all = a.tokens * a.top, s0 = blockIdx.x * each;
    for (int64_t s = s0 + threadIdx.x; s < s0 + each && s < all; s += kThreads) {
        const int e = a.chosen[s];
        if (e >= 0 && e < a.experts) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kThreads) a.counts[(int64_t)blockIdx.x * a.experts + e] = hist[e];
}

// Slots sorted by expert, those of one expert in their own order.  Each block
// sums the counts of all blocks (its own first places, every expert's first
// one), then walks its slots in order, a wave a quarter of them; lanes with one
// expert find each other by the bits of its number.
__global__ __launch_bounds__(kThreads) void plan_kernel(PlanArgs a) {
    extern __shared__ int next[];  // [kWaves][E], then [E + 1]
    __shared__ int part[kThreads];
    const int E = a.experts, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    int *first = next + kWaves * E;
    const int64_t each = (int64_t)a.block_tokens * a.top, all = a.tokens * a.top;
    const int64_t b0 = blockIdx.x * each, b1 = b0 + each < all ? b0 + each : all;
    const int64_t quarter = ((each + kWaves - 1) / kWaves + 63) / 64 * 64;
    const int64_t s0 = b0 + wave * quarter < b1 ? b0 + wave * quarter : b1, s1 = s0 + quarter < b1 ? s0 + quarter : b1;
    for (int i = threadIdx.x; i < kWaves * E; i += kThreads) next[i] = 0;
    __syncthreads();
    for (int64_t s = s0 + lane; s < s1; s += 64) {
        const int e = a.chosen[s];
        if (e >= 0 && e < E) atomicAdd(&next[wave * E + e], 1);
    }
    // (a thread's experts are neighbours)
    const int n = (E + kThreads - 1) / kThreads, e0 = threadIdx.x * n;
    int sum = 0;
    for (int e = e0; e < e0 + n && e < E; ++e) {
        int before = 0, total = 0;
        for (uint32_t b = 0; b < gridDim.x; ++b) {
            const int c = a.counts[(int64_t)b * E + e];
            before += b < blockIdx.x ? c : 0;
            total += c;
        }
        first[e] = before;
        sum += total;
    }
    part[threadIdx.x] = sum;
    __syncthreads();
    for (int o = 1; o < kThreads; o <<= 1) {
        const int v = (int)threadIdx.x >= o ? part[threadIdx.x - o] : 0;
        __syncthreads();
        part[threadIdx.x] += v;
        __syncthreads();
    }
    int at = part[threadIdx.x] - sum;
    const int used = part[kThreads - 1];
    for (int e = e0; e < e0 + n && e < E; ++e) {
        int total = 0;
        for (uint32_t b = 0; b < gridDim.x; ++b) total += a.counts[(int64_t)b * E + e];
        if (blockIdx.x == 0) a.offsets[e] = at;
        int p = at + first[e];
        for (int w = 0; w < kWaves; ++w) {
            const int c = next[w * E + e];
            next[w * E + e] = p;
            p += c;
        }
        at += total;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[E] = used;
    __syncthreads();
    const int bits = 32 - __builtin_clz(E);
    for (int64_t base = s0; base < s1; base += 64) {
        const int64_t s = base + lane;
        const int e = s < s1 ? a.chosen[s] : -1;
        const bool some = e >= 0 && e < E;
        uint64_t same = __ballot(some);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((e >> b) & 1);
            same &= (e >> b) & 1 ? set : ~set;
        }
        if (some) {
            const int rank = __popcll(same & ((1ull << lane) - 1));
            const int p = next[wave * E + e] + rank;
            a.place[s] = p;
            a.order[p] = (int)s;
        } else if (s < s1) {
            a.place[s] = -1;
        }
        // (every lane has read before the last of each expert counts on)
        __builtin_amdgcn_wave_barrier();
        if (some && (same >> lane) == 1) next[wave * E + e] += __popcll(same);
        __builtin_amdgcn_wave_barrier();
    }
    for (int64_t s = used + (int64_t)blockIdx.x * kThreads + threadIdx.x; s < all; s += (int64_t)gridDim.x * kThreads)
        a.order[s] = -1;
}

template <int NV>
__global__ __launch_bounds__(kThreads) void route_back_kernel(RouteBackArgs a, int G) {
    const int E = a.experts, lane = threadIdx.x & 63, gl = lane & (G - 1), first_lane = lane - gl;
    const int per = kThreads / G, own = threadIdx.x / G;
    for (int64_t base = (int64_t)blockIdx.x * per; base < a.tokens; base += (int64_t)gridDim.x * per) {
        const int64_t t = base + own;
        const bool live = t < a.tokens;
        int e = -1;
        float g = 0.0f, z = -INFINITY;
        if (live && gl < a.top) {
            e = a.chosen[t * a.top + gl];
            if (e < 0 || e >= E) e = -1;
            if (e >= 0) {
                g = a.scale * a.dweights[t * a.top + gl];
                z = read_logit(a.logits, t * a.ld + e, a.bf16);
            }
        }
        float v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = 0.0f;
        float d = 0.0f;
        if (a.renormalise) {
            const float l = e < 0 ? -INFINITY : a.sigmoid ? log_logistic(z) : z;
            const float m = group_max(l, G), x = e < 0 ? 0.0f : expf(l - m);
            const float s = group_sum(x, G), w = e < 0 ? 0.0f : x / s;
            const float dot = group_sum(w * g, G);
            d = w * (g - dot);
            if (a.sigmoid) d *= logistic(-z);
        } else if (a.sigmoid) {
            d = g * logistic(z) * logistic(-z);
        } else {
            float r[NV], top = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int x = gl + G * i;
                r[i] = live && x < E ? read_logit(a.logits, t * a.ld + x, a.bf16) : -INFINITY;
                top = fmaxf(top, r[i]);
            }
            top = group_max(top, G);
            const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                v[i] = r[i] == -INFINITY ? 0.0f : expf(r[i] - ref);
                sum += v[i];
            }
            sum = group_sum(sum, G);
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            const float p = e < 0 ? 0.0f : expf(z - ref) * inv;
            const float dot = group_sum(e < 0 ? 0.0f : p * g, G);
            d = p * g;
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] *= -inv * dot;
        }
        for (int j = 0; j < a.top; ++j) {
            const int x = __shfl(e, first_lane + j);
            const float y = __shfl(d, first_lane + j);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (x >= 0 && x == gl + G * i) v[i] += y;
        }
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int x = gl + G * i;
                if (x >= E) continue;
                if (a.bf16)
                    reinterpret_cast<uint16_t *>(a.dlogits)[t * a.lddl + x] = (uint16_t)tg_pack_bf16(v[i], 0.0f);
                else
                    reinterpret_cast<float *>(a.dlogits)[t * a.lddl + x] = v[i];
            }
        }
    }
}

int lanes(int experts) {
    int g = 1;
    while (g < experts && g < 64) g <<= 1;
    return g;
}
int64_t blocks_of(int64_t tokens, int32_t each) { return (tokens + each - 1) / each; }

}  // namespace

int32_t route_block_tokens(int64_t tokens, int32_t top) {
    const int64_t most = 256;
    int64_t each = (tokens + most - 1) / most;
    const int64_t least = (256 + top - 1) / top;
    return (int32_t)(each < least ? least : each);
}

hipError_t launch_route(const RouteArgs &a, hipStream_t stream) {
    const int G = lanes(a.experts), nv = (a.experts + G - 1) / G, per = kThreads / G;
    const size_t lds = (size_t)((a.experts + 1) / 2 + (a.groups > 1 ? per * (a.experts + a.groups) : 0)) * 8;
    const dim3 grid((uint32_t)blocks_of(a.tokens, a.block_tokens)), block(kThreads);
    if (nv == 1) hipLaunchKernelGGL(route_kernel<1>, grid, block, lds, stream, a, G);
    else if (nv == 2) hipLaunchKernelGGL(route_kernel<2>, grid, block, lds, stream, a, G);
    else if (nv <= 4) hipLaunchKernelGGL(route_kernel<4>, grid, block, lds, stream, a, G);
    else if (nv <= 8) hipLaunchKernelGGL(route_kernel<8>, grid, block, lds, stream, a, G);
    else hipLaunchKernelGGL(route_kernel<16>, grid, block, lds, stream, a, G);
    return hipGetLastError();
}

hipError_t launch_plan_count(const PlanArgs &a, hipStream_t stream) {
    hipLaunchKernelGGL(plan_count_kernel, dim3((uint32_t)blocks_of(a.tokens, a.block_tokens)), dim3(kThreads),
                       a.experts * 4, stream, a);
    return hipGetLastError();
}

hipError_t launch_plan(const PlanArgs &a, hipStream_t stream) {
    hipLaunchKernelGGL(plan_kernel, dim3((uint32_t)blocks_of(a.tokens, a.block_tokens)), dim3(kThreads),
                       (kWaves + 1) * a.experts * 4, stream, a);
    return hipGetLastError();
}

hipError_t launch_route_back(const RouteBackArgs &a, hipStream_t stream) {
    const int G = lanes(a.experts), nv = (a.experts + G - 1) / G, per = kThreads / G;
    const int64_t blocks = (a.tokens + per - 1) / per;
    const dim3 grid((uint32_t)(blocks < (1 << 20) ? blocks : 1 << 20)), block(kThreads);
    if (nv == 1) hipLaunchKernelGGL(route_back_kernel<1>, grid, block, 0, stream, a, G);
    else if (nv == 2) hipLaunchKernelGGL(route_back_kernel<2>, grid, block, 0, stream, a, G);
    else if (nv <= 4) hipLaunchKernelGGL(route_back_kernel<4>, grid, block, 0, stream, a, G);
    else if (nv <= 8) hipLaunchKernelGGL(route_back_kernel<8>, grid, block, 0, stream, a, G);
    else hipLaunchKernelGGL(route_back_kernel<16>, grid, block, 0, stream, a, G);
    return hipGetLastError();
}

}  // namespace zopt
