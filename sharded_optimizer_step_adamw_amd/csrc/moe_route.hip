// moe_route.hip -- routing of tokens to experts: scores, choice, weights, the
// slots' order by expert, and the logits' gradient.
#include <cmath>
#include <type_traits>

#include "lanes.h"
#include "moe_internal.h"

namespace zopt {
namespace {

constexpr int kRouteThreads = 512, kPlanThreads = 256, kAloneThreads = 1024;
// One block, in one launch, instead of several and three launches, which also cost the host
// 6 us more.  Measured with the host ahead, one block and three launches, us:
//   the choice and the sort, in two rounds of what a block chooses at once   7.1 and 9.9 (8
//   experts), 9.4 and 11.7 (64), with ranks of scores 10.4 and 11.8, 12.7 and 13.2; in four
//   9.9 and 10.5, 14.5 and 11.6, with ranks of scores 16.4 and 12.2, 20.9 and 13.3
//   the sort alone   4096 slots of 8 to 512 experts 7.0 to 9.1 and 8.3 to 9.7, 8192 10.0 to
//   13.6 and 8.4 to 9.8; 1024 slots of 1024 experts, by 256 threads, 7.9 and 10.5, 2048
//   11.4 and 10.7
constexpr int kRounds = 4, kScoredRounds = 2;
constexpr int64_t kAloneSlots = 4096, kManyExpertsSlots = 2048;
constexpr int kAloneExperts = 512;

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

__device__ __forceinline__ float logistic(float z) {
    const float e = expf(-fabsf(z));
    return (z >= 0.0f ? 1.0f : e) / (1.0f + e);
}
// What weights are in proportion to, of a logit z among the chosen ones, whose
// largest is m: its exponential or logistic, both times a power of e that keeps the
// largest near 1 however small they are (0 beside a NaN, whose own is one).
__device__ __forceinline__ float proportion(float z, float m, bool sigmoid) {
    if (!sigmoid) return expf(z - m);
    return (z >= 0.0f ? 1.0f : expf(z - fminf(m, 0.0f))) / (1.0f + expf(-fabsf(z)));
}

// Ranks as whole numbers in the same order: 0 for -inf (an expert that is not
// there), 1 for NaN, -0 as 0.
__device__ __forceinline__ uint32_t rank_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    const uint32_t r = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return v != v ? 1u : v == -INFINITY ? 0u : r;
}
// The value of a rank above 1.
__device__ __forceinline__ float value_of(uint32_t r) {
    return __uint_as_float(r ^ ((uint32_t)((int32_t)~r >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint64_t rank_of(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    const uint64_t r = b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
    return v != v ? 1ull : v == -(double)INFINITY ? 0ull : r;
}

struct RouteLane {
    int gl, first, row;  // the lane's number of its token's G, the first of them, the token's number in the block
};

// (what lanes of one wave have written to LDS, read by others of it)
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Whether a range of experts is a power of two of whole lanes.
__host__ __device__ __forceinline__ bool even_ranges(int experts, int groups, int G, int nv) {
    const int size = experts / groups, lanes = size / nv;
    return lanes * nv == size && (lanes & (lanes - 1)) == 0 && experts == G * nv;
}

struct BestTwo {
    float b1, b2;
    __device__ __forceinline__ void add(float k) {
        b2 = k > b1 ? b1 : k > b2 ? k : b2;
        b1 = k > b1 ? k : b1;
    }
    __device__ __forceinline__ float sum() const { return b2 == -INFINITY ? b1 : b1 + b2; }
};

// The ranges' sums of their two best; -inf to the experts of all but the best
// top_groups.  Returns how near that choice was: the last sum chosen less the
// first one left (inf: none was left).  lds: of the token, its ranges' sums and,
// where ranges are not even, the experts' keys.
template <int NV, int G>
__device__ __forceinline__ float choose_ranges(const RouteArgs &a, const RouteLane &l, float (&key)[NV], float *sums) {
    const int size = a.experts / a.groups, lanes = size / NV, e0 = l.gl * NV;
    // (a NaN's place behind every number; two of them are still a number)
    auto order = [](float v) __attribute__((always_inline)) { return v != v ? -1.5e38f : v; };
    float last = INFINITY, left = -INFINITY;
    // whether range x, of sum v, stays
    auto stays = [&](float v, int x) __attribute__((always_inline)) {
        int n = 0;
        for (int h = 0; h < a.groups; ++h) {
            const float s = sums[h];
            n += s > v || (s == v && h < x) ? 1 : 0;
        }
        const bool in = n < a.top_groups;
        last = in && v < last ? v : last;
        left = !in && v > left ? v : left;
        return in;
    };
    if (even_ranges(a.experts, a.groups, G, NV)) {
        BestTwo two{-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < NV; ++i) two.add(order(key[i]));
        two = join(two, lanes, [](BestTwo x, BestTwo y) {
            return BestTwo{fmaxf(x.b1, y.b1), fmaxf(fminf(x.b1, y.b1), fmaxf(x.b2, y.b2))};
        });
        const int g = l.gl / lanes;
        if (l.gl % lanes == 0) sums[g] = two.sum();
        wave_sync();
        const bool in = stays(two.sum(), g);
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = in ? key[i] : -INFINITY;
    } else {
        float *keys = sums + a.groups;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (e0 + i < a.experts) keys[e0 + i] = order(key[i]);
        wave_sync();
        for (int x = l.gl; x < a.groups; x += G) {
            BestTwo two{-INFINITY, -INFINITY};
            for (int i = 0; i < size; ++i) two.add(keys[x * size + i]);
            sums[x] = two.sum();
        }
        wave_sync();
        int at = -1;
        bool in = false;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (e0 + i >= a.experts) continue;
            if ((e0 + i) / size != at) {
                at = (e0 + i) / size;
                in = stays(sums[at], at);
            }
            key[i] = in ? key[i] : -INFINITY;
        }
    }
    wave_sync();
    last = join(last, G, [](float x, float y) { return fminf(x, y); });
    left = group_fmax(left, G);
    return left == -INFINITY ? INFINITY : last - left;
}

// The best `count` experts, one after the other, the j-th returned in lane j (-1:
// none is left): the best rank of all lanes, the lowest lane that has it, its
// lowest expert of that rank.
template <int NV, int G>
__device__ __forceinline__ int choose(const RouteLane &l, uint32_t (&rank)[NV], int count) {
    int chosen = -1;
    constexpr uint64_t lanes = G == 64 ? ~0ull : (1ull << (G & 63)) - 1;
    for (int j = 0; j < count; ++j) {
        uint32_t best = rank[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < NV; ++i) {
            at = rank[i] > best ? i : at;
            best = rank[i] > best ? rank[i] : best;
        }
        const uint32_t top = group_max(best, G);
        const uint64_t have = (__ballot(best == top) >> l.first) & lanes;
        const int lead = __builtin_ctzll(have);
        const int e = __shfl(l.gl * NV + at, l.first + lead);
        if (l.gl == j) chosen = top != 0 ? e : -1;
        const int gone = l.gl == lead ? at : -1;
#pragma unroll
        for (int i = 0; i < NV; ++i) rank[i] = gone == i ? 0 : rank[i];
    }
    return chosen;
}

// The choice of one token in 64 bits, by a whole wave: the j-th best expert
// returned in lane j.  lds: [experts + groups], the wave's.  It runs for few
// tokens, mostly not yet in the instruction cache: loops are short.
__device__ __forceinline__ int choose_exactly(const RouteArgs &a, int64_t t, double *lds) {
    const int lane = threadIdx.x & 63, E = a.experts;
    constexpr double kNone = -INFINITY;
    uint64_t *keys = reinterpret_cast<uint64_t *>(lds);
    float top = -INFINITY;
#pragma unroll 4
    for (int e = lane; e < E; e += 64) {
        const float z = read_logit(a.logits, t * a.ld + e, a.bf16);
        lds[e] = (double)z;
        top = fmaxf(top, z);
    }
    double total = 1.0, ref = 0.0;
    if (!a.sigmoid) {
        top = group_fmax(top, 64);
        ref = top == -INFINITY ? 0.0 : (double)top;
        total = 0.0;
#pragma unroll 1
        for (int e = lane; e < E; e += 64) total += exp(lds[e] - ref);
        total = group_sum(total, 64);
    }
#pragma unroll 1
    for (int e = lane; e < E; e += 64) {
        const double z = lds[e], x = exp(a.sigmoid ? -z : z - ref);
        double k = (a.sigmoid ? 1.0 : x) / (a.sigmoid ? 1.0 + x : total);
        const double b = a.bias != nullptr ? (double)a.bias[e] : 0.0;
        k += b;
        lds[e] = fmin(z, b) == kNone ? kNone : k != k ? -0.85e308 : k;  // (as in choose_ranges)
    }
    wave_sync();
    if (a.groups > 1) {
        const int size = E / a.groups;
        double b1 = kNone, b2 = kNone;
        if (lane < a.groups) {
#pragma unroll 4
            for (int i = 0; i < size; ++i) {
                const double k = lds[lane * size + i];
                b2 = k > b1 ? b1 : k > b2 ? k : b2;
                b1 = k > b1 ? k : b1;
            }
            b1 = b2 == kNone ? b1 : b1 + b2;
            lds[E + lane] = b1;
        }
        wave_sync();
        int before = 0;
#pragma unroll 4
        for (int h = 0; h < a.groups; ++h) {
            const double s = lds[E + h];
            before += s > b1 || (s == b1 && h < lane) ? 1 : 0;
        }
        const uint64_t in = __ballot(lane < a.groups && before < a.top_groups);
#pragma unroll 1
        for (int e = lane; e < E; e += 64)
            if (!((in >> (e / size)) & 1)) lds[e] = kNone;
        wave_sync();
    }
#pragma unroll 1
    for (int e = lane; e < E; e += 64) keys[e] = rank_of(lds[e]);
    int chosen = -1;
#pragma unroll 1
    for (int j = 0; j < a.top; ++j) {
        uint64_t best = 0;
        int at = 0x7FFFFFFF;
#pragma unroll 4
        for (int e = lane; e < E; e += 64) {
            const uint64_t k = keys[e];
            at = k > best ? e : at;
            best = k > best ? k : best;
        }
        const uint64_t most = group_max(best, 64);
        at = join(best == most ? at : 0x7FFFFFFF, 64, [](int x, int y) { return x < y ? x : y; });
        if (lane == j) chosen = most != 0 ? at : -1;
        if (most != 0 && (at & 63) == lane) keys[at] = 0;
    }
    wave_sync();
    return chosen;
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
// formed in fp32 first.  With steps of 2^-24, a score p is off by
//   logistic   p times 4 (the exponential; over all arguments 1.4) + 1 + 1 (1 + it, the
//              quotient): 6 (2.8)
//   softmax    p times d (the rounding of its logit's distance d to the largest) + 4 (the
//              exponential) + 4 + 7 (the sum, kept in 64 bits, of terms that are off so,
//              whose mean distance is below the logarithm of 1024 experts) + 1 + 1: d + 17
// and a rank by one step of its own besides (all of them with 2^-8 more, for what is of the
// second order); below fp32's range, or where an exponential overflows, by 2^-126.  No
// distance past 128 counts, of which no score is left.
// Then the chosen ones are looked at again, the logistic's scores in 64 bits: each has
// to lie before the next, by more than both may be off if they are not of the same
// logit and bias, and the last before all that are left, each with what it may be off
// itself: one far down the order may have a large score and a bias that takes it away,
// and so be off by more than the best one left.  That is asked for the largest rank left
// and the largest score there can be first, and expert by expert in waves with a token
// where that does not settle it.
// A token where all that does not hold is ranked again in 64 bits throughout, by the
// whole wave: one of 16384 makes the launch 1 us longer.
// Bound by instruction issue and latency (16384 tokens over 256 experts in 8
// groups, 16.8 MB: 35 us; 40 with 4 experts a lane, and 55 held to 80 registers for
// more waves).
template <int NV, int G>
__global__ __launch_bounds__(kRouteThreads, 4) void route_kernel(RouteArgs a, PlanArgs plan) {
    extern __shared__ double lds[];
    const int E = a.experts, waves = blockDim.x / 64;
    double *exact = lds + (threadIdx.x >> 6) * (E + a.groups);
    float *rows = reinterpret_cast<float *>(lds + (a.scored ? waves * (E + a.groups) : 0));
    int *hist = reinterpret_cast<int *>(rows + blockDim.x / G * a.row_floats);
    const int lane = threadIdx.x & 63, per = blockDim.x / G;
    const RouteLane l{lane & (G - 1), lane & ~(G - 1), (int)threadIdx.x / G};
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * a.block_tokens;
    const int64_t t1 = t0 + a.block_tokens < a.tokens ? t0 + a.block_tokens : a.tokens;
    for (int64_t base = t0; base < t1; base += per) {
        const int64_t t = base + l.row;
        const bool live = t < t1;
        float z[NV];
        read_logits<NV>(a.logits, t * a.ld + l.gl * NV, live ? E - l.gl * NV : 0, a.bf16, z);
        uint32_t rank[NV];
        float top = -INFINITY, ref = 0.0f, sum = 1.0f;
        float key[NV];
        if (!a.sigmoid && (a.scored || !a.renormalise)) {
#pragma unroll
            for (int i = 0; i < NV; ++i) top = fmaxf(top, z[i]);
            top = group_fmax(top, G);
            ref = top == -INFINITY ? 0.0f : top;
            double total = 0.0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                key[i] = expf(z[i] - ref);
                total += (double)key[i];
            }
            sum = (float)group_sum(total, G);
        }
        bool near = false;
        int expert;
        float zc = -INFINITY;  // the lane's expert's logit
        if (a.scored) {
            auto score = [&](float z, float e) __attribute__((always_inline)) {
                return a.sigmoid ? 1.0f / (1.0f + expf(-z)) : e / sum;
            };
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = l.gl * NV + i;
                const float b = a.bias != nullptr && e < E ? a.bias[e] : 0.0f;
                key[i] = fminf(z[i], b) == -INFINITY ? -INFINITY : score(z[i], key[i]) + b;
            }
            if (a.groups > 1) {
#pragma unroll
                for (int i = 0; i < NV; ++i) near |= fabsf(key[i]) > 2.0f && key[i] != -INFINITY;
                const float gap = choose_ranges<NV, G>(a, l, key, rows + l.row * a.row_floats);
                // (Two sums of two ranks that are 2 at most.  Logistic scores: 4 x 6 steps, 4 x 2 of the
                // ranks and 2 x 4 of the sums, 40 in all; a softmax's scores are together 1 at
                // most and p d below 1 / e, 19 + 16.)
                near |= !(gap > 0x1p-18f);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) rank[i] = rank_of(key[i]);
            expert = choose<NV, G>(l, rank, a.top);
            // (d: how far its logit lies below the largest)
            auto may_be_off = [&](float p, float d, float rank) __attribute__((always_inline)) {
                return 0x1.01p-24f * (p * (a.sigmoid ? 6.0f : 17.0f + fminf(d, 128.0f)) + fabsf(rank)) + 0x1p-126f;
            };
            float bc = 0.0f;
            double exactly = -INFINITY, off = 0.0;  // the rank again, and how far it may be off
            if (expert >= 0) {
                zc = read_logit(a.logits, t * a.ld + expert, a.bf16);
                bc = a.bias != nullptr ? a.bias[expert] : 0.0f;
                const float p = score(zc, a.sigmoid ? 0.0f : expf(zc - ref)), about = p + bc;
                exactly = a.sigmoid ? 1.0 / (1.0 + exp(-(double)zc)) + (double)bc : (double)about;
                off = a.sigmoid ? 0.0 : (double)may_be_off(p, ref - zc, about);
                near |= about != about;
            }
            const double before = __shfl_up(exactly, 1), before_off = __shfl_up(off, 1);
            const bool same = __shfl_up(zc, 1) == zc && __shfl_up(bc, 1) == bc;
            near |= l.gl > 0 && l.gl < a.top && expert >= 0 && !(before - exactly > before_off + off || same);
            // The last chosen against what is left.  (Ranks as numbers are in the order of
            // rank + 2^-24 |rank|, too, and e^-d (d + 17) is largest for d = 0; fewer chosen
            // than `top`: nothing is left.)
            uint32_t most = rank[0];
#pragma unroll
            for (int i = 1; i < NV; ++i) most = rank[i] > most ? rank[i] : most;
            most = group_max(most, G);
            const bool last = l.gl == a.top - 1 && expert >= 0 && most > 1;
            const double least = exactly - off;
            const float left = value_of(most);
            const bool unclear = last && !(least > (double)left + (double)may_be_off(a.sigmoid ? 1.0f : 1.0f / sum, 0.0f, left));
            if (__ballot(unclear) != 0) {
                const float zl = __shfl(zc, l.first + a.top - 1), bl = __shfl(bc, l.first + a.top - 1);
                double worst = -INFINITY;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    // (one expert after the other: few registers; an equal of the last one lies behind it)
                    __builtin_amdgcn_sched_barrier(0);
                    if (rank[i] <= 1) continue;
                    const int e = l.gl * NV + i;
                    const float z = read_logit(a.logits, t * a.ld + e, a.bf16), b = a.bias != nullptr ? a.bias[e] : 0.0f;
                    const float p = score(z, a.sigmoid ? 0.0f : expf(z - ref)), about = value_of(rank[i]);
                    const double most = (double)about + (double)may_be_off(p, ref - z, about);
                    worst = (z != zl || b != bl) && most > worst ? most : worst;
                }
                worst = join(worst, G, [](double x, double y) { return x > y ? x : y; });
                near |= unclear && !(least > worst);
            }
            uint64_t again = __ballot(near && live);
            while (again != 0) {
                // the lowest token of those, by all lanes
                const int first = __builtin_ctzll(again) & ~(G - 1);
                const int exactly = choose_exactly(a, base + (threadIdx.x - lane + first) / G, exact);
                const int mine = __shfl(exactly, l.gl);
                if (l.first == first) {
                    expert = mine;
                    zc = expert >= 0 ? read_logit(a.logits, t * a.ld + expert, a.bf16) : -INFINITY;
                }
                again &= ~((G == 64 ? ~0ull : (1ull << (G & 63)) - 1) << first);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) rank[i] = rank_of(z[i]);
            expert = choose<NV, G>(l, rank, a.top);
            if (expert >= 0) zc = read_logit(a.logits, t * a.ld + expert, a.bf16);
        }
        const bool picked = expert >= 0 && l.gl < a.top;
        float w = 0.0f;
        if (a.renormalise) {
            const float m = group_fmax(picked ? zc : -INFINITY, G), e = picked ? proportion(zc, m, a.sigmoid) : 0.0f;
            const float s = group_sum(e, G);
            w = picked ? a.scale * (e / s) : 0.0f;
        } else if (picked) {
            w = a.scale * (a.sigmoid ? logistic(zc) : expf(zc - top) / sum);
        }
        if (live && l.gl < a.top) {
            a.chosen[t * a.top + l.gl] = picked ? expert : -1;
            a.weights[t * a.top + l.gl] = w;
            if (picked && gridDim.x > 1) atomicAdd(&hist[expert], 1);
        }
    }
    __syncthreads();
    if (a.sort_here) {
        __threadfence_block();
        __syncthreads();
        sort_block<kRouteThreads>(plan, 0, 1, nullptr, nullptr, reinterpret_cast<int *>(lds));
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

template <int THREADS>
__global__ __launch_bounds__(THREADS) void plan_kernel(PlanArgs a) {
    extern __shared__ int next[];
    const bool alone = gridDim.x == 1;
    sort_block<THREADS>(a, blockIdx.x, gridDim.x, alone ? nullptr : a.counts + (int64_t)blockIdx.x * a.experts,
                             alone ? nullptr : a.total, next);
}

template <int NV, int G>
__global__ __launch_bounds__(256) void route_back_kernel(RouteBackArgs a) {
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
            const float m = group_fmax(z, G), x = e < 0 ? 0.0f : proportion(z, m, a.sigmoid);
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

// Lanes of a token, 4 or more and as many as the experts chosen at least, and experts of
// a lane: 8 from 128 experts on, else 4 (and 16 where a wave's lanes do not do).
// Choosing 8 of 128 for 16384 tokens takes 11.4 us with 8, 13.8 with 4; 6 of 60 for
// 4099 7.3 with 4.
struct Lanes {
    int G, nv;
};
Lanes lanes_of(int experts, int top) {
    const int each = experts < 128 ? 4 : 8;
    int g = 4;
    while (g < 64 && (g * each < experts || g < top)) g <<= 1;
    return {g, experts <= 4 * g ? 4 : experts <= 8 * g ? 8 : 16};
}
// f<NV, G>()
template <class F>
void with_lanes(Lanes l, F f) {
    using std::integral_constant;
    if (l.nv == 16) f(integral_constant<int, 16>{}, integral_constant<int, 64>{});
    else if (l.nv == 8 && l.G == 64) f(integral_constant<int, 8>{}, integral_constant<int, 64>{});
    else if (l.nv == 8 && l.G == 32) f(integral_constant<int, 8>{}, integral_constant<int, 32>{});
    else if (l.nv == 8) f(integral_constant<int, 8>{}, integral_constant<int, 16>{});
    else if (l.G == 64) f(integral_constant<int, 4>{}, integral_constant<int, 64>{});
    else if (l.G == 32) f(integral_constant<int, 4>{}, integral_constant<int, 32>{});
    else if (l.G == 16) f(integral_constant<int, 4>{}, integral_constant<int, 16>{});
    else if (l.G == 8) f(integral_constant<int, 4>{}, integral_constant<int, 8>{});
    else f(integral_constant<int, 4>{}, integral_constant<int, 4>{});
}
int64_t blocks_of(int64_t tokens, int32_t each) { return (tokens + each - 1) / each; }

// LDS of the choice with `threads` a block: the waves' for the choice in 64 bits,
// the tokens' for their ranges, the experts' counts
int32_t route_row(int32_t experts, int32_t groups, int32_t top) {
    const Lanes l = lanes_of(experts, top);
    return groups == 1 ? 0 : even_ranges(experts, groups, l.G, l.nv) ? groups : groups + experts;
}
size_t route_lds(int32_t experts, int32_t groups, int32_t top, bool scored, int threads) {
    return (size_t)(scored ? threads / 64 * (experts + groups) * 8 : 0) +
           (size_t)(threads / lanes_of(experts, top).G * route_row(experts, groups, top) + experts) * 4;
}
constexpr size_t kRouteLds = 48 << 10;

}  // namespace

int32_t route_block_tokens(int64_t tokens, int32_t experts, int32_t groups, int32_t top, bool scored) {
    const int64_t at_once = experts > 0 ? kRouteThreads / lanes_of(experts, top).G : 0;
    const bool one = experts < 0 ? tokens * top <= (-experts <= kAloneExperts ? kAloneSlots : kManyExpertsSlots)
                                 : tokens <= (scored ? kScoredRounds : kRounds) * at_once &&
                                       route_lds(experts, groups, top, scored, kRouteThreads) <= kRouteLds;
    if (one) return (int32_t)(tokens > 0 ? tokens : 1);
    // at most 1024 blocks, of 256 slots or of what a block chooses at once or more
    const int64_t each = (tokens + 1023) / 1024, least = experts > 0 ? at_once : (256 + top - 1) / top;
    return (int32_t)(each < least ? least : each);
}

hipError_t launch_route(RouteArgs a, const PlanArgs &plan, hipStream_t stream) {
    const Lanes l = lanes_of(a.experts, a.top);
    const uint32_t blocks = (uint32_t)blocks_of(a.tokens, a.block_tokens);
    const int threads =
        route_lds(a.experts, a.groups, a.top, a.scored, kRouteThreads) <= kRouteLds ? kRouteThreads : 256;
    const size_t choice = route_lds(a.experts, a.groups, a.top, a.scored, threads);
    a.sort_here = blocks == 1 && threads == kRouteThreads;
    a.row_floats = route_row(a.experts, a.groups, a.top);
    const size_t sort = a.sort_here ? (size_t)(kRouteThreads / 64 + 1) * a.experts * 4 : 0;
    const size_t bytes = choice > sort ? choice : sort;
    with_lanes(l, [&](auto NV, auto G) {
        hipLaunchKernelGGL((route_kernel<decltype(NV)::value, decltype(G)::value>), dim3(blocks), dim3(threads), bytes,
                           stream, a, plan);
    });
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
    if (blocks == 1 && a.tokens * a.top > kPlanThreads && a.experts <= kAloneExperts)
        hipLaunchKernelGGL(plan_kernel<kAloneThreads>, dim3(1), dim3(kAloneThreads), (kAloneThreads / 64 + 1) * a.experts * 4,
                           stream, a);
    else
        hipLaunchKernelGGL(plan_kernel<kPlanThreads>, dim3((uint32_t)(blocks > 0 ? blocks : 1)), dim3(kPlanThreads),
                           (kPlanThreads / 64 + 1) * a.experts * 4, stream, a);
    return hipGetLastError();
}

hipError_t launch_route_back(const RouteBackArgs &a, hipStream_t stream) {
    const Lanes l = lanes_of(a.experts, a.top);
    const int per = 256 / l.G;
    const int64_t blocks = (a.tokens + per - 1) / per;
    with_lanes(l, [&](auto NV, auto G) {
        hipLaunchKernelGGL((route_back_kernel<decltype(NV)::value, decltype(G)::value>),
                           dim3((uint32_t)(blocks < (1 << 20) ? blocks : 1 << 20)), dim3(256), 0, stream, a);
    });
    return hipGetLastError();
}

}  // namespace zopt
