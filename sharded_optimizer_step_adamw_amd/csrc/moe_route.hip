// moe_route.hip -- routing of tokens to experts: scores, choice, weights, the
// slots' order by expert, and the logits' gradient.
#include <cmath>

#include "lanes.h"
#include "moe_internal.h"

namespace zopt {
namespace {

constexpr int kRouteThreads = 512, kPlanThreads = 256;
// A grid of one block chooses and sorts in one launch.
constexpr int64_t kOneBlockSlots = 2048;

// ------------------------------------------------------------------ scores

__device__ __forceinline__ float read_logit(const void *p, int64_t i, bool bf16) {
    return bf16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p)[i] << 16)
                : reinterpret_cast<const float *>(p)[i];
}
// NV neighbouring logits of a row from e on, -inf behind the last
template <int NV>
__device__ __forceinline__ void read_logits(const void *p, int64_t i, int left, bool bf16, float (&z)[NV]) {
    if (left >= NV && NV >= 4) {
        if (bf16) {
#pragma unroll
            for (int k = 0; k < NV; k += 4) {
                const tg_u32x2 r = tg_load<tg_u32x2>(reinterpret_cast<const uint16_t *>(p) + i + k);
                z[k] = __uint_as_float(r.x << 16);
                z[k + 1] = __uint_as_float(r.x & 0xFFFF0000u);
                z[k + 2] = __uint_as_float(r.y << 16);
                z[k + 3] = __uint_as_float(r.y & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int k = 0; k < NV; k += 4) {
                const tg_f32x4 r = tg_load<tg_f32x4>(reinterpret_cast<const float *>(p) + i + k);
#pragma unroll
                for (int m = 0; m < 4; ++m) z[k + m] = r[m];
            }
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) z[k] = k < left ? read_logit(p, i + k, bf16) : -INFINITY;
}

// log of the logistic function, and the function
__device__ __forceinline__ float log_logistic(float z) { return fminf(z, 0.0f) - log1pf(expf(-fabsf(z))); }
__device__ __forceinline__ float logistic(float z) {
    const float e = expf(-fabsf(z));
    return (z >= 0.0f ? 1.0f : e) / (1.0f + e);
}

// Ranks as whole numbers in the same order: 0 for -inf (an expert that is not
// there), 1 for NaN, -0 as 0.
__device__ __forceinline__ uint32_t rank_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    const uint32_t r = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return v != v ? 1u : v == -INFINITY ? 0u : r;
}
__device__ __forceinline__ uint64_t rank_of(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    const uint64_t r = b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
    return v != v ? 1ull : v == -(double)INFINITY ? 0ull : r;
}

struct RouteLane {
    int G, gl, first, row;  // lanes of a token, the lane's number there, its first lane, the token's number in the block
};

// Two-best sums of the ranges of experts, and -inf to the experts of all but
// the best top_groups.  Returns how near the choice of ranges was: the sum of
// the last one chosen less that of the first one left (inf: no choice).
template <int NV, class R>
__device__ __forceinline__ R choose_ranges(const RouteArgs &a, const RouteLane &l, R (&key)[NV], double *lds) {
    const int size = a.experts / a.groups, lanes = size / NV;
    const R kNone = -(R)INFINITY;
    auto order = [](R v) __attribute__((always_inline)) { return v != v ? (R)-3.0e38f : v; };
    R own = kNone;
    int g = 0, groups = a.groups;
    // (the token's own LDS in both types: its neighbours' may be in use in the other one)
    R *sums = reinterpret_cast<R *>(lds + (int64_t)l.row * (a.experts + a.groups)) + a.experts;
    if (lanes * NV == size && (lanes & (lanes - 1)) == 0 && a.experts == l.G * NV) {
        // a range is a power of two of lanes
        struct Two {
            R b1, b2;
        } two{kNone, kNone};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const R k = order(key[i]);
            two.b2 = k > two.b1 ? two.b1 : k > two.b2 ? k : two.b2;
            two.b1 = k > two.b1 ? k : two.b1;
        }
        two = join(two, lanes, [](Two x, Two y) {
            const R lo = x.b1 < y.b1 ? x.b1 : y.b1, hi = x.b2 > y.b2 ? x.b2 : y.b2;
            return Two{x.b1 > y.b1 ? x.b1 : y.b1, lo > hi ? lo : hi};
        });
        own = two.b2 == kNone ? two.b1 : two.b1 + two.b2;
        g = l.gl / lanes;
        if (l.gl % lanes == 0) sums[g] = own;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    } else {
        R *keys = sums - a.experts;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (l.gl * NV + i < a.experts) keys[l.gl * NV + i] = order(key[i]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        for (int x = l.gl; x < groups; x += l.G) {
            R b1 = kNone, b2 = kNone;
            for (int i = 0; i < size; ++i) {
                const R k = keys[x * size + i];
                b2 = k > b1 ? b1 : k > b2 ? k : b2;
                b1 = k > b1 ? k : b1;
            }
            sums[x] = b2 == kNone ? b1 : b1 + b2;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        g = -1;
    }
    R last = (R)INFINITY, left = kNone;
    auto before = [&](R v, int x) __attribute__((always_inline)) {
        int n = 0;
        for (int h = 0; h < groups; ++h) {
            const R s = sums[h];
            n += s > v || (s == v && h < x) ? 1 : 0;
        }
        return n;
    };
    auto stays = [&](R v, int x) __attribute__((always_inline)) {
        const bool in = before(v, x) < a.top_groups;
        if (in) last = v < last ? v : last;
        else left = v > left ? v : left;
        return in;
    };
    if (g >= 0) {
        const bool in = stays(own, g);
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = in ? key[i] : kNone;
    } else {
        int at = -1;
        bool in = false;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = l.gl * NV + i;
            if (e >= a.experts) continue;
            if (e / size != at) {
                at = e / size;
                in = stays(sums[at], at);
            }
            key[i] = in ? key[i] : kNone;
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    last = join(last, l.G, [](R x, R y) { return x < y ? x : y; });
    left = group_max(left, l.G);
    return left == kNone ? (R)INFINITY : last - left;
}

// What lane j of a token knows of its j-th best expert.
struct Pick {
    int expert;       // -1: none
    float z, bias, key;
};

// The best `count` experts, one after the other: the best rank of all lanes,
// the lowest lane that has it, its lowest expert of that rank.
template <int NV, class K>
__device__ __forceinline__ Pick choose(const RouteLane &l, K (&rank)[NV], const float (&z)[NV], const float (&bias)[NV],
                                       const float (&key)[NV], int count) {
    Pick p{-1, 0.0f, 0.0f, 0.0f};
    const uint64_t lanes = l.G == 64 ? ~0ull : (1ull << l.G) - 1;
    for (int j = 0; j < count; ++j) {
        K best = rank[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < NV; ++i) {
            at = rank[i] > best ? i : at;
            best = rank[i] > best ? rank[i] : best;
        }
        const K top = group_max(best, l.G);
        const uint64_t have = (__ballot(best == top) >> l.first) & lanes;
        const int lead = __builtin_ctzll(have);
        float zi = z[0], bi = bias[0], ki = key[0];
#pragma unroll
        for (int i = 1; i < NV; ++i) {
            zi = at == i ? z[i] : zi;
            bi = at == i ? bias[i] : bi;
            ki = at == i ? key[i] : ki;
        }
        const int from = l.first + lead;
        const int e = __shfl(l.gl * NV + at, from);
        zi = __shfl(zi, from);
        if (l.gl == j) {
            p.expert = top != 0 ? e : -1;
            p.z = zi;
        }
        if (sizeof(K) == 4) {
            bi = __shfl(bi, from);
            ki = __shfl(ki, from);
            if (l.gl == j) {
                p.bias = bi;
                p.key = ki;
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) rank[i] = l.gl == lead && at == i ? 0 : rank[i];
    }
    return p;
}

// Sorts the slots of block `block` of `blocks`: base [experts], how many slots
// of each expert lie in the blocks before (NULL: none do); total [experts], in
// all of them (NULL: this one's own).  Each wave walks a part of the slots in
// order; lanes with one expert find each other by the bits of its number.
// next: LDS, [waves + 1][experts].
// (THREADS: the block's)
template <int THREADS>
__device__ __forceinline__ void sort_block(const PlanArgs &a, int block, int blocks, const int32_t *base,
                                           const int32_t *total, int *next) {
    constexpr int kWaves = THREADS / 64;
    __shared__ int part[THREADS];
    const int E = a.experts, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t each = (int64_t)a.block_tokens * a.top, all = a.tokens * a.top;
    const int64_t b0 = block * each, b1 = b0 + each < all ? b0 + each : all;
    const int64_t share = ((each + kWaves - 1) / kWaves + 63) / 64 * 64;
    const int64_t s0 = b0 + wave * share < b1 ? b0 + wave * share : b1, s1 = s0 + share < b1 ? s0 + share : b1;
    for (int i = threadIdx.x; i < kWaves * E; i += THREADS) next[i] = 0;
    __syncthreads();
    for (int64_t s = s0 + lane; s < s1; s += 64) {
        const int e = a.chosen[s];
        if (e >= 0 && e < E) atomicAdd(&next[wave * E + e], 1);
    }
    __syncthreads();
    // (a thread's experts are neighbours)
    const int n = (E + THREADS - 1) / THREADS, e0 = threadIdx.x * n, e1 = e0 + n < E ? e0 + n : E;
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        int c = 0;
        if (total != nullptr) c = total[e];
        else
            for (int w = 0; w < kWaves; ++w) c += next[w * E + e];
        next[kWaves * E + e] = c;
        sum += c;
    }
    part[threadIdx.x] = sum;
    __syncthreads();
    for (int o = 1; o < THREADS; o <<= 1) {
        const int v = (int)threadIdx.x >= o ? part[threadIdx.x - o] : 0;
        __syncthreads();
        part[threadIdx.x] += v;
        __syncthreads();
    }
    int at = part[threadIdx.x] - sum;
    const int used = part[THREADS - 1];
    for (int e = e0; e < e1; ++e) {
        if (block == 0) a.offsets[e] = at;
        int p = at + (base != nullptr ? base[e] : 0);
        for (int w = 0; w < kWaves; ++w) {
            const int c = next[w * E + e];
            next[w * E + e] = p;
            p += c;
        }
        at += next[kWaves * E + e];
    }
    if (block == 0 && threadIdx.x == 0) a.offsets[E] = used;
    __syncthreads();
    const int bits = 32 - __builtin_clz(E);
    for (int64_t s = s0 + lane; s - lane < s1; s += 64) {
        const int e = s < s1 ? a.chosen[s] : -1;
        const bool some = e >= 0 && e < E;
        uint64_t same = __ballot(some);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((e >> b) & 1);
            same &= (e >> b) & 1 ? set : ~set;
        }
        if (some) {
            const int p = next[wave * E + e] + __popcll(same & ((1ull << lane) - 1));
            a.place[s] = p;
            a.order[p] = (int)s;
        } else if (s < s1) {
            a.place[s] = -1;
        }
        // (every lane has read before the last of each expert counts on)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (some && (same >> lane) == 1) next[wave * E + e] += __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    for (int64_t s = used + (int64_t)block * THREADS + threadIdx.x; s < all; s += (int64_t)blocks * THREADS)
        a.order[s] = -1;
}

// G lanes a token, NV neighbouring experts a lane.  Ranks by score and bias are
// formed in fp32 first, off by less than 2^-19 (1 + |rank|): the sum of at most
// 16 6-fold joined exponentials by 22 2^-24 of itself, each exponential,
// quotient and the bias's addition by some 2^-24 more.  Where two of the best
// lie closer than that could hide, and are not of the same logit and bias, the
// wave's tokens are ranked again in 64 bits.
template <int NV>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a, PlanArgs plan, int G) {
    extern __shared__ double lds[];
    const int E = a.experts;
    int *hist = reinterpret_cast<int *>(lds);
    double *keys = lds + (E + 1) / 2;
    const int lane = threadIdx.x & 63, per = blockDim.x / G;
    const RouteLane l{G, lane & (G - 1), lane & ~(G - 1), (int)threadIdx.x / G};
    const bool scored = a.bias != nullptr || a.groups > 1;
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * a.block_tokens;
    const int64_t t1 = t0 + a.block_tokens < a.tokens ? t0 + a.block_tokens : a.tokens;
    float bias[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = l.gl * NV + i;
        bias[i] = a.bias != nullptr && e < E ? a.bias[e] : 0.0f;
    }
    for (int64_t base = t0; base < t1; base += per) {
        const int64_t t = base + l.row;
        const bool live = t < t1;
        float z[NV], key[NV];
        read_logits<NV>(a.logits, t * a.ld + l.gl * NV, live ? E - l.gl * NV : 0, a.bf16, z);
        float top = -INFINITY, sum = 0.0f;
        if (!a.sigmoid && (scored || !a.renormalise)) {
#pragma unroll
            for (int i = 0; i < NV; ++i) top = fmaxf(top, z[i]);
            top = group_fmax(top, G);
            const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                key[i] = __expf(z[i] - ref);
                sum += key[i];
            }
            sum = group_sum(sum, G);
        }
        uint32_t rank[NV];
        bool near = false;
        Pick p;
        if (scored) {
            const float inv = 1.0f / sum;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float s = a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + __expf(-z[i])) : key[i] * inv;
                key[i] = z[i] == -INFINITY ? -INFINITY : s + bias[i];
            }
            if (a.groups > 1) {
                const float gap = choose_ranges<NV, float>(a, l, key, keys);
                near = !(gap > 0x1p-15f);  // (of sums of two, each rank below 2 in size)
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                rank[i] = rank_of(key[i]);
                near |= fabsf(key[i]) > 2.0f && key[i] != -INFINITY && a.groups > 1;
            }
            p = choose<NV>(l, rank, z, bias, key, a.top + 1);
            // against the one before
            const float before = __shfl_up(p.key, 1), zb = __shfl_up(p.z, 1), bb = __shfl_up(p.bias, 1);
            const int eb = __shfl_up(p.expert, 1);
            if (l.gl > 0 && l.gl <= a.top && p.expert >= 0 && eb >= 0) {
                const bool apart = before - p.key > 0x1p-18f * (1.0f + fmaxf(fabsf(before), fabsf(p.key)));
                near |= !apart && !(zb == p.z && bb == p.bias);
            }
            near |= p.key != p.key;
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) rank[i] = rank_of(z[i]);
            p = choose<NV>(l, rank, z, bias, z, a.top);
        }
        if (__any(near)) {
            const bool again = group_max(near ? 1 : 0, G) != 0;
            double wide[NV], total = 0.0;
            if (!a.sigmoid) {
                const double ref = top == -INFINITY ? 0.0 : (double)top;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    wide[i] = z[i] == -INFINITY ? 0.0 : exp((double)z[i] - ref);
                    total += wide[i];
                }
                total = group_sum(total, G);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)z[i])) : wide[i] / total;
                wide[i] = z[i] == -INFINITY ? -(double)INFINITY : s + (double)bias[i];
            }
            if (a.groups > 1) choose_ranges<NV, double>(a, l, wide, keys);
            uint64_t wide_rank[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) wide_rank[i] = rank_of(wide[i]);
            const Pick q = choose<NV>(l, wide_rank, z, bias, z, a.top);
            if (again) p = q;
        }
        const bool picked = p.expert >= 0 && l.gl < a.top;
        float w = 0.0f;
        if (a.renormalise) {
            const float x = !picked ? -INFINITY : a.sigmoid ? log_logistic(p.z) : p.z;
            const float m = group_fmax(x, G), e = picked ? expf(x - m) : 0.0f;
            const float s = group_sum(e, G);
            w = picked ? a.scale * (e / s) : 0.0f;
        } else if (picked) {
            w = a.scale * (a.sigmoid ? logistic(p.z) : expf(p.z - top) / sum);
        }
        if (live && l.gl < a.top) {
            a.chosen[t * a.top + l.gl] = p.expert;
            a.weights[t * a.top + l.gl] = w;
            if (picked && gridDim.x > 1) atomicAdd(&hist[p.expert], 1);
        }
    }
    __syncthreads();
    if (a.sort_here) {
        __threadfence_block();
        __syncthreads();
        sort_block<kRouteThreads>(plan, 0, 1, nullptr, nullptr, hist);
        return;
    }
    // (one block's slots are counted where they are sorted)
    if (gridDim.x == 1) return;
    for (int e = threadIdx.x; e < E; e += blockDim.x) plan.counts[(int64_t)blockIdx.x * E + e] = hist[e];
}

__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(PlanArgs a) {
    extern __shared__ int hist[];
    for (int e = threadIdx.x; e < a.experts; e += kPlanThreads) hist[e] = 0;
    __syncthreads();
    const int64_t each = (int64_t)a.block_tokens * a.top, all = a.tokens * a.top, s0 = blockIdx.x * each;
    for (int64_t s = s0 + threadIdx.x; s < s0 + each && s < all; s += kPlanThreads) {
        const int e = a.chosen[s];
        if (e >= 0 && e < a.experts) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kPlanThreads) a.counts[(int64_t)blockIdx.x * a.experts + e] = hist[e];
}

// counts [blocks, experts] to what lies in the blocks before, their sums to
// total.  A block takes 16 experts, a thread every 64th block of one.
__global__ __launch_bounds__(1024) void plan_scan_kernel(PlanArgs a, int blocks) {
    __shared__ int part[64][17];
    const int e = blockIdx.x * 16 + (threadIdx.x & 15), r = threadIdx.x >> 4;
    const int each = (blocks + 63) / 64, b0 = r * each, b1 = b0 + each < blocks ? b0 + each : blocks;
    const bool live = e < a.experts;
    int32_t *p = a.counts + e;
    int sum = 0;
    if (live) {
#pragma unroll 8
        for (int b = b0; b < b1; ++b) sum += p[(int64_t)b * a.experts];
    }
    part[r][threadIdx.x & 15] = sum;
    __syncthreads();
    if (r == 0) {
        int at = 0;
        for (int k = 0; k < 64; ++k) {
            const int c = part[k][threadIdx.x];
            part[k][threadIdx.x] = at;
            at += c;
        }
        if (live) a.total[e] = at;
    }
    __syncthreads();
    int at = part[r][threadIdx.x & 15];
    if (live) {
#pragma unroll 8
        for (int b = b0; b < b1; ++b) {
            const int c = p[(int64_t)b * a.experts];
            p[(int64_t)b * a.experts] = at;
            at += c;
        }
    }
}

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanArgs a) {
    extern __shared__ int next[];
    const bool alone = gridDim.x == 1;
    sort_block<kPlanThreads>(a, blockIdx.x, gridDim.x, alone ? nullptr : a.counts + (int64_t)blockIdx.x * a.experts,
                             alone ? nullptr : a.total, next);
}

template <int NV>
__global__ __launch_bounds__(256) void route_back_kernel(RouteBackArgs a, int G) {
    const int E = a.experts, lane = threadIdx.x & 63, gl = lane & (G - 1), first_lane = lane - gl, e0 = gl * NV;
    const int per = 256 / G, own = threadIdx.x / G;
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
            const float m = group_fmax(l, G), x = e < 0 ? 0.0f : expf(l - m);
            const float s = group_sum(x, G), w = e < 0 ? 0.0f : x / s;
            const float dot = group_sum(w * g, G);
            d = w * (g - dot);
            if (a.sigmoid) d *= logistic(-z);
        } else if (a.sigmoid) {
            d = g * logistic(z) * logistic(-z);
        } else {
            float r[NV], top = -INFINITY, sum = 0.0f;
            read_logits<NV>(a.logits, t * a.ld + e0, live ? E - e0 : 0, a.bf16, r);
#pragma unroll
            for (int i = 0; i < NV; ++i) top = fmaxf(top, r[i]);
            top = group_fmax(top, G);
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
            const int x = __shfl(e, first_lane + j) - e0;
            const float y = __shfl(d, first_lane + j);
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] += x == i ? y : 0.0f;
        }
        if (!live) continue;
        const int64_t at = t * a.lddl + e0;
        if (NV >= 4 && e0 + NV <= E) {
#pragma unroll
            for (int i = 0; i < NV; i += 4) {
                if (a.bf16)
                    tg_store(reinterpret_cast<uint16_t *>(a.dlogits) + at + i,
                             tg_u32x2{tg_pack_bf16(v[i], v[i + 1]), tg_pack_bf16(v[i + 2], v[i + 3])});
                else
                    tg_store(reinterpret_cast<float *>(a.dlogits) + at + i, tg_f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]});
            }
            continue;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (e0 + i >= E) continue;
            if (a.bf16)
                reinterpret_cast<uint16_t *>(a.dlogits)[at + i] = (uint16_t)tg_pack_bf16(v[i], 0.0f);
            else
                reinterpret_cast<float *>(a.dlogits)[at + i] = v[i];
        }
    }
}

// Lanes of a token: one for four experts, more than the experts chosen, at
// most a wave; and experts of a lane.
struct Lanes {
    int G, nv;
};
Lanes lanes_of(int experts, int top) {
    int g = 1;
    while (g < 64 && (g * 4 < experts || g <= top)) g <<= 1;
    int nv = 1;
    while (nv * g < experts) nv <<= 1;
    return {g, nv};
}
int64_t blocks_of(int64_t tokens, int32_t each) { return (tokens + each - 1) / each; }

// LDS of the choice with `threads` a block
size_t route_lds(int32_t experts, int32_t groups, int32_t top, int threads) {
    const int64_t rows = groups > 1 ? threads / lanes_of(experts, top).G : 0;
    return (size_t)((experts + 1) / 2 + rows * (experts + groups)) * 8;
}
constexpr size_t kRouteLds = 48 << 10;

}  // namespace

int32_t route_block_tokens(int64_t tokens, int32_t experts, int32_t groups, int32_t top) {
    const int64_t at_once = experts > 0 ? kRouteThreads / lanes_of(experts, top).G : 0;
    if (tokens * top <= kOneBlockSlots &&
        (experts == 0 || (tokens <= 4 * at_once && route_lds(experts, groups, top, kRouteThreads) <= kRouteLds)))
        return (int32_t)(tokens > 0 ? tokens : 1);
    // at most 1024 blocks, of 256 slots or of what a block chooses at once or more
    const int64_t each = (tokens + 1023) / 1024, least = experts > 0 ? at_once : (256 + top - 1) / top;
    return (int32_t)(each < least ? least : each);
}

hipError_t launch_route(RouteArgs a, const PlanArgs &plan, hipStream_t stream) {
    const Lanes l = lanes_of(a.experts, a.top);
    const uint32_t blocks = (uint32_t)blocks_of(a.tokens, a.block_tokens);
    const int threads = route_lds(a.experts, a.groups, a.top, kRouteThreads) <= kRouteLds ? kRouteThreads : 256;
    const size_t choice = route_lds(a.experts, a.groups, a.top, threads);
    a.sort_here = blocks == 1 && threads == kRouteThreads;
    const size_t sort = a.sort_here ? (size_t)(kRouteThreads / 64 + 1) * a.experts * 4 : 0;
    const size_t bytes = choice > sort ? choice : sort;
    const dim3 grid(blocks), block(threads);
    if (l.nv == 1) hipLaunchKernelGGL(route_kernel<1>, grid, block, bytes, stream, a, plan, l.G);
    else if (l.nv == 2) hipLaunchKernelGGL(route_kernel<2>, grid, block, bytes, stream, a, plan, l.G);
    else if (l.nv == 4) hipLaunchKernelGGL(route_kernel<4>, grid, block, bytes, stream, a, plan, l.G);
    else if (l.nv == 8) hipLaunchKernelGGL(route_kernel<8>, grid, block, bytes, stream, a, plan, l.G);
    else hipLaunchKernelGGL(route_kernel<16>, grid, block, bytes, stream, a, plan, l.G);
    hipError_t e = hipGetLastError();
    return e == hipSuccess && !a.sort_here ? launch_plan(plan, stream) : e;
}

hipError_t launch_plan_count(const PlanArgs &a, hipStream_t stream) {
    const int64_t blocks = blocks_of(a.tokens, a.block_tokens);
    if (blocks == 1) return hipSuccess;
    hipLaunchKernelGGL(plan_count_kernel, dim3((uint32_t)blocks), dim3(kPlanThreads), a.experts * 4, stream, a);
    return hipGetLastError();
}

hipError_t launch_plan(const PlanArgs &a, hipStream_t stream) {
    const int64_t blocks = blocks_of(a.tokens, a.block_tokens);
    if (blocks > 1) {
        hipLaunchKernelGGL(plan_scan_kernel, dim3((uint32_t)((a.experts + 15) / 16)), dim3(1024), 0, stream, a,
                           (int)blocks);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(plan_kernel, dim3((uint32_t)(blocks > 0 ? blocks : 1)), dim3(kPlanThreads),
                       (kPlanThreads / 64 + 1) * a.experts * 4, stream, a);
    return hipGetLastError();
}

hipError_t launch_route_back(const RouteBackArgs &a, hipStream_t stream) {
    const Lanes l = lanes_of(a.experts, a.top);
    const int per = 256 / l.G;
    const int64_t blocks = (a.tokens + per - 1) / per;
    const dim3 grid((uint32_t)(blocks < (1 << 20) ? blocks : 1 << 20)), block(256);
    if (l.nv == 1) hipLaunchKernelGGL(route_back_kernel<1>, grid, block, 0, stream, a, l.G);
    else if (l.nv == 2) hipLaunchKernelGGL(route_back_kernel<2>, grid, block, 0, stream, a, l.G);
    else if (l.nv == 4) hipLaunchKernelGGL(route_back_kernel<4>, grid, block, 0, stream, a, l.G);
    else if (l.nv == 8) hipLaunchKernelGGL(route_back_kernel<8>, grid, block, 0, stream, a, l.G);
    else hipLaunchKernelGGL(route_back_kernel<16>, grid, block, 0, stream, a, l.G);
    return hipGetLastError();
}

}  // namespace zopt
