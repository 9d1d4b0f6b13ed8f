// lanes.h -- maxima and sums over aligned groups of 1, 2, 4, ... 64 lanes of a
// wave (gfx950), in registers.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace zopt {
namespace {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
// v of the lanes whose values f joins with the own one's, step by step: after
// log2(G) steps every lane of G has the result.  (A mirror instead of an
// exchange does as well: the lanes that it passes over agree by then.)
template <class T, class F>
__device__ __forceinline__ T join(T v, int G, F f) {
    constexpr int kWords = sizeof(T) / 4;
    union Words {
        T t;
        uint32_t w[kWords];
    };
    auto step = [&](auto move) __attribute__((always_inline)) {
        Words x;
        x.t = v;
#pragma unroll
        for (int k = 0; k < kWords; ++k) x.w[k] = move(x.w[k]);
        v = f(v, x.t);
    };
    if (G >= 2) step([](uint32_t x) { return dpp<0xB1>(x); });   // lanes ^ 1
    if (G >= 4) step([](uint32_t x) { return dpp<0x4E>(x); });   // lanes ^ 2
    if (G >= 8) step([](uint32_t x) { return dpp<0x141>(x); });  // mirrored in 8
    if (G >= 16) step([](uint32_t x) { return dpp<0x140>(x); }); // mirrored in 16
    const int lane = threadIdx.x & 63;
    if (G >= 32)
        step([&](uint32_t x) {
            const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
            return lane & 16 ? r[0] : r[1];
        });
    if (G >= 64)
        step([&](uint32_t x) {
            const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
            return lane & 32 ? r[0] : r[1];
        });
    return v;
}
template <class T>
__device__ __forceinline__ T group_max(T v, int G) {
    return join(v, G, [](T a, T b) { return a > b ? a : b; });
}
__device__ __forceinline__ float group_fmax(float v, int G) {
    return join(v, G, [](float a, float b) { return fmaxf(a, b); });
}
template <class T>
__device__ __forceinline__ T group_sum(T v, int G) {
    return join(v, G, [](T a, T b) { return a + b; });
}

}  // namespace
}  // namespace zopt
