// moe_rows.hip -- the passes over rows around the experts' products: tokens
// gathered by expert, the tile rows of experts whose sizes only the device
// knows, and the sums over a token's experts.  All are bound by HBM.
#include "lanes.h"
#include "moe_internal.h"
#include "tile_walk.h"

namespace zopt {
namespace {

constexpr int kThreads = 256;

uint32_t blocks_for(int64_t n) {
    const int64_t b = (n + kThreads - 1) / kThreads;
    return (uint32_t)(b < 1 ? 1 : b > (1 << 20) ? (1 << 20) : b);
}

// A value of the routing's arrays as an index in [0, n], whatever was given:
// arrays that are not a routing's give wrong sums, but no access out of range.
__device__ __forceinline__ int within(int v, int64_t n) { return v < 0 ? 0 : v > n ? (int)n : v; }

// Expert e's rows
__device__ __forceinline__ void bounds(const MoePrepList &l, int e, int &lo, int &n) {
    lo = within(l.offsets[e], l.slots);
    const int hi = within(l.offsets[e + 1], l.slots);
    n = hi > lo ? hi - lo : 0;
}

// Counts that stop at 2^30: offsets that are no routing's may count every slot for
// every expert.
__device__ __forceinline__ int more(int a, int b) {
    const uint32_t s = (uint32_t)a + (uint32_t)b;  // (both at most 2^30)
    return (int)(s < (1u << 30) ? s : 1u << 30);
}

__device__ __forceinline__ void prep_tiles(const MoePrepList &l, const MoePrep &j) {
    __shared__ int at[kMaxExperts];
    __shared__ int part[kThreads];
    constexpr int kEach = kMaxExperts / kThreads;
    int lo, n, sum = 0;
    // (a thread's experts are neighbours)
    for (int i = 0; i < kEach; ++i) {
        const int e = threadIdx.x * kEach + i;
        if (e >= l.experts) break;
        bounds(l, e, lo, n);
        sum += (n + j.height - 1) / j.height;
    }
    part[threadIdx.x] = sum;
    __syncthreads();
    for (int o = 1; o < kThreads; o <<= 1) {
        const int v = (int)threadIdx.x >= o ? part[threadIdx.x - o] : 0;
        __syncthreads();
        part[threadIdx.x] = more(part[threadIdx.x], v);
        __syncthreads();
    }
    int first = part[threadIdx.x] - sum;
    for (int i = 0; i < kEach; ++i) {
        const int e = threadIdx.x * kEach + i;
        if (e >= l.experts) break;
        at[e] = first;
        bounds(l, e, lo, n);
        first += (n + j.height - 1) / j.height;
    }
    if (threadIdx.x == 0) {
        const int all = part[kThreads - 1];
        j.tiles[0] = TgTileRow{all < j.capacity ? all : j.capacity, 0, 0, 0};
    }
    __syncthreads();
    const int lane = threadIdx.x & 63;
    for (int e = threadIdx.x >> 6; e < l.experts; e += kThreads / 64) {
        bounds(l, e, lo, n);
        const int all = (n + j.height - 1) / j.height, left = j.capacity - at[e];
        for (int r = lane; r < all && r < left; r += 64)
            j.tiles[1 + at[e] + r] = TgTileRow{e, lo + r * j.height, lo + n, 0};
    }
}

// How many parts expert e has (1: it is whole), and how many rows each
__device__ __forceinline__ int parts_of(int n, int most, int &rows) {
    const int parts = n <= most ? 1 : (n + most - 1) / most;
    rows = parts == 1 ? n : ((n + parts - 1) / parts + 63) / 64 * 64;
    return parts == 1 ? 1 : (n + rows - 1) / rows;
}
__device__ __forceinline__ void prep_items(const MoePrepList &l, const MoePrep &j) {
    __shared__ int size[kMaxExperts];
    __shared__ int part[2][kThreads];
    constexpr int kEach = kMaxExperts / kThreads;
    int lo, n, rows, sum = 0, split = 0;
    for (int i = 0; i < kEach; ++i) {
        const int e = threadIdx.x * kEach + i;
        if (e >= l.experts) break;
        bounds(l, e, lo, n);
        const int parts = parts_of(n, j.height, rows);
        size[e] = parts > 1 ? -1 : n;
        sum += parts > 1 ? parts : 0;
        split += parts > 1 ? 1 : 0;
    }
    part[0][threadIdx.x] = sum;
    part[1][threadIdx.x] = split;
    __syncthreads();
    for (int o = 1; o < kThreads; o <<= 1) {
        const int v = (int)threadIdx.x >= o ? part[0][threadIdx.x - o] : 0;
        const int w = (int)threadIdx.x >= o ? part[1][threadIdx.x - o] : 0;
        __syncthreads();
        part[0][threadIdx.x] = more(part[0][threadIdx.x], v);
        part[1][threadIdx.x] += w;
        __syncthreads();
    }
    const int parts = part[0][kThreads - 1], joins = part[1][kThreads - 1];
    // (more than a routing's offsets give: offsets that are none, and no items)
    const bool wrong = parts > 2 * (l.slots / j.height) || joins > l.slots / j.height;
    if (threadIdx.x == 0) j.tiles[0] = wrong ? TgItem{0, 0, 0, 0} : TgItem{parts + l.experts - joins, parts, joins, 0};
    if (wrong) return;
    int at = part[0][threadIdx.x] - sum, join = part[1][threadIdx.x] - split;
    for (int i = 0; i < kEach; ++i) {
        const int e = threadIdx.x * kEach + i;
        if (e >= l.experts) break;
        bounds(l, e, lo, n);
        const int own = parts_of(n, j.height, rows);
        if (own == 1) continue;
        j.joins[join++] = TgItem{e, at, at + own, 0};
        for (int p = 0; p < own; ++p) {
            const int end = (p + 1) * rows < n ? (p + 1) * rows : n;
            j.tiles[1 + at++] = TgItem{e, lo + p * rows, lo + end, 0};
        }
    }
    // the others by size: tiles that run together then take about the same time
    for (int e = threadIdx.x; e < l.experts; e += kThreads) {
        if (size[e] < 0) continue;
        int rank = 0;
        for (int i = 0; i < l.experts; ++i) rank += size[i] > size[e] || (size[i] == size[e] && i < e) ? 1 : 0;
        bounds(l, e, lo, n);
        j.tiles[1 + parts + rank] = TgItem{e, lo, lo + n, 0};
    }
}

// A wave four times 1 KiB of a row, so that what leads to a row is read once for
// them: 16 bytes a thread took half as long again.
constexpr int kGatherPieces = 4 * 64;
__device__ __forceinline__ void prep_gather(const MoePrepList &l, const MoePrep &j, int64_t block) {
    const int64_t per = (j.cols + 7) / 8, chunks = (per + kGatherPieces - 1) / kGatherPieces;
    const int64_t total = within(l.offsets[l.experts], l.slots) * chunks;
    const int lane = threadIdx.x & 63;
    for (int64_t id = (block * kThreads + threadIdx.x) >> 6; id < total; id += (int64_t)j.blocks * (kThreads / 64)) {
        const int64_t s = id / chunks, c0 = (id - s * chunks) * kGatherPieces + lane;
        const int slot = l.order[s];
        const bool some = slot >= 0 && slot < l.slots;
        const uint16_t *from = j.src + (int64_t)(some ? slot / l.top : 0) * j.ld;
        uint16_t *to = j.dst + s * per * 8;
        tg_u32x4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = c0 + i * 64;
            v[i] = tg_u32x4{0, 0, 0, 0};
            if (some && c < per) v[i] = tg_load8h(from + c * 8, j.cols - c * 8 > 8 ? 8 : (int)(j.cols - c * 8));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = c0 + i * 64;
            if (c < per) *reinterpret_cast<tg_u32x4 *>(to + c * 8) = v[i];
        }
    }
}

__device__ __forceinline__ void prep_shares(const MoePrepList &l, const MoePrep &j, int64_t block) {
    for (int64_t s = block * kThreads + threadIdx.x; s < l.slots; s += (int64_t)j.blocks * kThreads) {
        const int slot = l.order[s];
        j.share[s] = slot >= 0 && slot < l.slots ? j.weights[slot] : 0.0f;
    }
}

__device__ __forceinline__ void prep_copy(const MoePrep &j, int64_t block) {
    const int64_t per = (j.cols + 7) / 8, total = j.rows * per;
    for (int64_t id = block * kThreads + threadIdx.x; id < total; id += (int64_t)j.blocks * kThreads) {
        const int64_t r = id / per, c = (id - r * per) * 8, left = j.cols - c, g = r / j.group_rows;
        *reinterpret_cast<tg_u32x4 *>(j.dst + id * 8) =
            tg_load8h(j.src + g * j.group_stride + (r - g * j.group_rows) * j.ld + c, left > 8 ? 8 : (int)left);
    }
}

__global__ __launch_bounds__(kThreads) void moe_prep_kernel(MoePrepList list) {
    uint32_t block = blockIdx.x;
    int k = 0;
    while (k + 1 < list.n && block >= list.job[k].blocks) block -= list.job[k++].blocks;
    const MoePrep &j = list.job[k];
    if (j.kind == kMoeTiles)
        prep_tiles(list, j);
    else if (j.kind == kMoeItems)
        prep_items(list, j);
    else if (j.kind == kMoeGather)
        prep_gather(list, j, block);
    else if (j.kind == kMoeShares)
        prep_shares(list, j, block);
    else
        prep_copy(j, block);
}

// Eight columns a thread; the sum over a token's slots in fp32, in their order.
__device__ __forceinline__ void combine_rows(const MoeCombine &c, int64_t block) {
    const int64_t per = (c.cols + 7) / 8, total = c.tokens * per;
    for (int64_t id = block * kThreads + threadIdx.x; id < total; id += (int64_t)c.sum_blocks * kThreads) {
        const int64_t t = id / per, col = (id - t * per) * 8, left = c.cols - col;
        float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
        for (int k = 0; k < c.top; ++k) {
            const int s = c.place[t * c.top + k];
            if (s < 0 || s >= c.slots) continue;
            const float w = c.weights != nullptr ? c.weights[t * c.top + k] : 1.0f;
            const tg_u32x4 r = *reinterpret_cast<const tg_u32x4 *>(c.rows + s * c.ld + col);
            const uint32_t e = c.scale[s * c.ldscale + col / kRowsGroup];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const tg_f16x2 h = __builtin_bit_cast(tg_f16x2, (uint32_t)r[i]);
                sum[2 * i] += w * tg_rows_out((float)h.x, e);
                sum[2 * i + 1] += w * tg_rows_out((float)h.y, e);
            }
        }
        tg_store8h(c.out + t * c.ldo + col, tg_pack8(sum), left > 8 ? 8 : (int)left);
    }
}

// The gradients of the tokens' weights: one wave a slot.
__device__ __forceinline__ void combine_dots(const MoeCombine &c, int64_t block) {
    const int lane = threadIdx.x & 63;
    for (int64_t i = (block * kThreads + threadIdx.x) >> 6; i < c.tokens * c.top;
         i += (int64_t)c.dot_blocks * (kThreads / 64)) {
        const int s = c.place[i];
        float sum = 0.0f;
        if (s >= 0 && s < c.slots)
            for (int p = lane; p < c.parts; p += 64) sum += c.dot[s * c.lddot + p];
        sum = group_sum(sum, 64);
        if (lane == 0) c.dweights[i] = sum;
    }
}

// A weight gradient's tiles that were summed in parts: a wave 16 rows of what one
// wave of the tile held, the parts added in order.
__device__ __forceinline__ void join_parts(const MoeJoin &j, int64_t block) {
    const TgLaunch &L = j.L;
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4, waves = j.rows * j.cols;
    const int blocks16 = j.height / j.rows / 16, per = L.tiles_m * L.tiles_n * L.nprob;
    const int64_t total = (int64_t)L.items[0].end * per * waves * blocks16;
    for (int64_t id = (block * kThreads + threadIdx.x) >> 6; id < total; id += (int64_t)j.blocks * (kThreads / 64)) {
        const int64_t tile = id / (waves * blocks16);
        const int wave = (int)(id / blocks16 % waves), i = (int)(id % blocks16), rest = (int)(tile % per);
        const TgItem join = L.joins[tile / per];
        const tg_f32x4 *p = reinterpret_cast<const tg_f32x4 *>(L.part) +
                            ((((int64_t)join.row * per + rest) * waves + wave) * blocks16 + i) * (4 * 64) + lane;
        tg_f32x4 acc[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = p[k * 64];
#pragma unroll 2
        for (int s = join.row + 1; s < join.end; ++s) {
            p += (int64_t)per * waves * blocks16 * (4 * 64);
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[k] += p[k * 64];
        }
        int prob, ti, tj;
        item_tile(L, rest, prob, ti, tj);
        const int row = ti * j.height + (wave / j.cols) * (blocks16 * 16) + i * 16 + c;
        const int col = tj * j.width + (wave % j.cols) * 64 + q * 4;
        if (row >= L.M) continue;
        uint16_t *o = L.prob[prob].out + join.group * L.group_out + row * L.ldc + col;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int left = L.N - col - k * 16;
            const tg_u32x2 v{tg_pack_bf16(acc[k][0], acc[k][1]), tg_pack_bf16(acc[k][2], acc[k][3])};
            if (left >= 4) {
                tg_store(o + k * 16, v);
            } else {
                if (left > 0) o[k * 16] = (uint16_t)v.x;
                if (left > 1) o[k * 16 + 1] = (uint16_t)(v.x >> 16);
                if (left > 2) o[k * 16 + 2] = (uint16_t)v.y;
            }
        }
    }
}

__global__ __launch_bounds__(kThreads) void moe_combine_kernel(MoeCombine c) {
    // (what has long chains of loads first)
    uint32_t block = blockIdx.x;
    if (block < c.join[0].blocks) return join_parts(c.join[0], block);
    block -= c.join[0].blocks;
    if (block < c.join[1].blocks) return join_parts(c.join[1], block);
    block -= c.join[1].blocks;
    if (block < c.dot_blocks) return combine_dots(c, block);
    combine_rows(c, block - c.dot_blocks);
}

__global__ __launch_bounds__(kThreads) void fill_zero_groups_kernel(uint16_t *dst, int64_t ld, int64_t group_stride,
                                                                    int64_t groups, int64_t rows, int64_t cols) {
    const int64_t each = rows * cols, total = groups * each;
    for (int64_t id = blockIdx.x * (int64_t)kThreads + threadIdx.x; id < total; id += (int64_t)gridDim.x * kThreads) {
        const int64_t g = id / each, r = (id - g * each) / cols;
        dst[g * group_stride + r * ld + (id - g * each - r * cols)] = 0;
    }
}

}  // namespace

hipError_t launch_moe_prep(MoePrepList &list, hipStream_t stream) {
    uint32_t total = 0;
    for (int k = 0; k < list.n; ++k) {
        MoePrep &j = list.job[k];
        const int64_t per = (j.cols + 7) / 8;
        j.blocks = j.kind == kMoeTiles || j.kind == kMoeItems ? 1
                   : j.kind == kMoeShares                     ? blocks_for(list.slots)
                   : j.kind == kMoeGather ? blocks_for(list.slots * ((per + kGatherPieces - 1) / kGatherPieces) * 64)
                                          : blocks_for(j.rows * per);
        total += j.blocks;
    }
    if (total == 0) return hipSuccess;
    hipLaunchKernelGGL(moe_prep_kernel, dim3(total), dim3(kThreads), 0, stream, list);
    return hipGetLastError();
}

hipError_t launch_moe_combine(MoeCombine &c, hipStream_t stream) {
    c.sum_blocks = blocks_for(c.tokens * ((c.cols + 7) / 8));
    c.dot_blocks = c.dweights != nullptr ? blocks_for(c.tokens * c.top * 64) : 0;
    for (MoeJoin &j : c.join) {
        // (how many groups have parts only the device knows: few blocks, which mostly
        // end at once)
        const int64_t waves = c.dweights != nullptr ? (int64_t)j.L.join_limit * j.L.tiles_m * j.L.tiles_n * j.L.nprob *
                                                          j.cols * (j.height / 16)
                                                    : 0;
        const int64_t blocks = (waves + 3) / 4;
        j.blocks = (uint32_t)(blocks < 1024 ? blocks : 1024);
    }
    hipLaunchKernelGGL(moe_combine_kernel, dim3(c.sum_blocks + c.dot_blocks + c.join[0].blocks + c.join[1].blocks),
                       dim3(kThreads), 0, stream, c);
    return hipGetLastError();
}

hipError_t launch_fill_zero_groups(uint16_t *dst, int64_t ld, int64_t group_stride, int64_t groups, int64_t rows,
                                   int64_t cols, hipStream_t stream) {
    hipLaunchKernelGGL(fill_zero_groups_kernel, dim3(blocks_for(groups * rows * cols)), dim3(kThreads), 0, stream, dst,
                       ld, group_stride, groups, rows, cols);
    return hipGetLastError();
}

}  // namespace zopt
