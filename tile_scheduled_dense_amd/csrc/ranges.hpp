// ranges.hpp -- host helpers of the C ABI's argument checks: address ranges and
// integer rounding.
#pragma once

#include <cstdint>

#include "tile_gemm.h"

namespace tg {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Byte extent [lo, hi) touched by a strided-batched row-major operand.
struct Range {
    uintptr_t lo, hi;
};

inline Range span(const void *p, int64_t batch, int64_t rows, int64_t cols, int64_t ld, int64_t stride, int esz) {
    if (batch == 0 || rows == 0 || cols == 0) return {0, 0};
    const uintptr_t base = reinterpret_cast<uintptr_t>(p);
    const int64_t last = (batch - 1) * stride + (rows - 1) * ld + cols;   // one past the last element
    return {base, base + static_cast<uintptr_t>(last) * esz};
}

inline bool overlaps(Range a, Range b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

// gfx950 check for the current device, cached per device (tile_gemm.hip).
tg_status device_ok();

}  // namespace tg
