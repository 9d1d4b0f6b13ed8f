// train_api.h -- what the entry points of the gradient operators share: their
// limits, the layout of a workspace, the checks of arguments.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "zopt.h"

#define ZOPT_EXPORT extern "C" __attribute__((visibility("default")))

namespace zopt {
namespace {

constexpr int64_t kMaxSide = 1 << 21;          // D, F, V: a 256-row panel stays below 2^31 bytes
constexpr int64_t kMaxRows = 1 << 30;          // T
constexpr int64_t kMaxStride = (1 << 22) - 8;  // of an operand read in place

inline int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// Offsets into a workspace, in order, 256-byte aligned.
struct Carve {
    size_t off = 0;
    size_t take(int64_t bytes) {
        const size_t at = off;
        off += (size_t)up(bytes, 256);
        return at;
    }
    size_t total() const { return off; }
};

inline size_t larger(size_t a, size_t b) { return a > b ? a : b; }

bool range(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }
bool stride_ok(int64_t ld, int64_t cols) { return ld >= cols && ld <= ((int64_t)1 << 31); }

zopt_status device(hipError_t e) { return e == hipSuccess ? ZOPT_OK : ZOPT_ERR_DEVICE; }
#define ZOPT_TRY(x)                                 \
    do {                                            \
        const hipError_t e_ = (x);                  \
        if (e_ != hipSuccess) return ZOPT_ERR_DEVICE; \
    } while (0)

zopt_status workspace_check(size_t need, void *workspace, size_t given) {
    if (given < need || ((uintptr_t)workspace & 255)) return ZOPT_ERR_WORKSPACE;
    return ZOPT_OK;
}

}  // namespace
}  // namespace zopt
