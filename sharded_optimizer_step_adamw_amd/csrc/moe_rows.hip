// moe_rows.hip -- the passes over rows around the experts' products: tokens
// gathered by expert, the tile rows of experts whose sizes only the device
// knows, and the sums over a token's experts.  All are bound by HBM.
#include "moe_internal.h"

namespace zopt {
namespace {

constexpr int kThreads = 256;

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

// A value of the routing's arrays as an index in [0, n], whatever was given:
// arrays that are not a routing's give wrong sums, but no access out of range.
__device__ __forceinline__ int within(int v, int64_t n) { return v < 0 ? 0 : v > n ? (int)n : v; }

// Expert e's rows
__device__ __forceinline__ void bounds(const MoePrepList &l, int e, int &lo, int &n) {
    lo = within(l.offsets[e], l.slots);
    const int hi = within(l.offsets[e + 1], l.slots);
    n = hi > lo ? hi - lo : 0;
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
        part[threadIdx.x] += v;
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
        for (int r = lane; r * j.height < n; r += 64)
            if (at[e] + r < j.capacity) j.tiles[1 + at[e] + r] = TgTileRow{e, lo + r * j.height, lo + n, 0};
    }
}

__device__ __forceinline__ void prep_sizes(const MoePrepList &l, const MoePrep &j) {
    __shared__ int size[kMaxExperts];
    int lo, n;
    for (int e = threadIdx.x; e < l.experts; e += kThreads) {
        bounds(l, e, lo, n);
        size[e] = n;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < l.experts; e += kThreads) {
        const int own = size[e];
        int rank = 0;
        for (int i = 0; i < l.experts; ++i) rank += size[i] > own || (size[i] == own && i < e) ? 1 : 0;
        j.sizes[rank] = e;
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

__device__ __forceinline__ void prep_tokens(const MoePrepList &l, const MoePrep &j, int64_t block) {
    for (int64_t s = block * kThreads + threadIdx.x; s < l.slots; s += (int64_t)j.blocks * kThreads) {
        const int slot = l.order[s];
        const bool some = slot >= 0 && slot < l.slots;
        j.token[s] = some ? slot / l.top : -1;
        if (j.share != nullptr) j.share[s] = some ? j.weights[slot] : 0.0f;
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
    else if (j.kind == kMoeSizes)
        prep_sizes(list, j);
    else if (j.kind == kMoeGather)
        prep_gather(list, j, block);
    else if (j.kind == kMoeTokens)
        prep_tokens(list, j, block);
    else
        prep_copy(j, block);
}

// Eight columns a thread; the sum over a token's slots in fp32, in their order.
__global__ __launch_bounds__(kThreads) void moe_combine_kernel(MoeCombine c) {
    const int64_t per = (c.cols + 7) / 8, total = c.tokens * per;
    for (int64_t id = blockIdx.x * (int64_t)kThreads + threadIdx.x; id < total; id += (int64_t)gridDim.x * kThreads) {
        const int64_t t = id / per, col = (id - t * per) * 8, left = c.cols - col;
        float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int k = 0; k < c.top; ++k) {
            const int s = c.place[t * c.top + k];
            if (s < 0 || s >= c.slots) continue;
            const float w = c.weights != nullptr ? c.weights[t * c.top + k] : 1.0f;
            float v[8];
            unpack8(*reinterpret_cast<const tg_u32x4 *>(c.rows + s * c.ld + col), v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += w * v[i];
        }
        tg_store8h(c.out + t * c.ldo + col, pack8(sum), left > 8 ? 8 : (int)left);
    }
}

// The gradients of the tokens' weights: one wave a slot.
__global__ __launch_bounds__(kThreads) void moe_dweights_kernel(MoeCombine c) {
    const int lane = threadIdx.x & 63;
    for (int64_t i = (blockIdx.x * (int64_t)kThreads + threadIdx.x) >> 6; i < c.tokens * c.top;
         i += (int64_t)gridDim.x * (kThreads / 64)) {
        const int s = c.place[i];
        float sum = 0.0f;
        if (s >= 0 && s < c.slots)
            for (int p = lane; p < c.parts; p += 64) sum += c.dot[s * c.lddot + p];
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
        if (lane == 0) c.dweights[i] = sum;
    }
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
        j.blocks = j.kind == kMoeTiles || j.kind == kMoeSizes ? 1
                   : j.kind == kMoeTokens                     ? blocks_for(list.slots)
                   : j.kind == kMoeGather ? blocks_for(list.slots * ((per + kGatherPieces - 1) / kGatherPieces) * 64)
                                          : blocks_for(j.rows * per);
        total += j.blocks;
    }
    if (total == 0) return hipSuccess;
    hipLaunchKernelGGL(moe_prep_kernel, dim3(total), dim3(kThreads), 0, stream, list);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeCombine &c, hipStream_t stream) {
    hipLaunchKernelGGL(moe_combine_kernel, dim3(blocks_for(c.tokens * ((c.cols + 7) / 8))), dim3(kThreads), 0, stream, c);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && c.dweights != nullptr) {
        hipLaunchKernelGGL(moe_dweights_kernel, dim3(blocks_for(c.tokens * c.top * 64)), dim3(kThreads), 0, stream, c);
        e = hipGetLastError();
    }
    return e;
}

hipError_t launch_fill_zero_groups(uint16_t *dst, int64_t ld, int64_t group_stride, int64_t groups, int64_t rows,
                                   int64_t cols, hipStream_t stream) {
    hipLaunchKernelGGL(fill_zero_groups_kernel, dim3(blocks_for(groups * rows * cols)), dim3(kThreads), 0, stream, dst,
                       ld, group_stride, groups, rows, cols);
    return hipGetLastError();
}

}  // namespace zopt
