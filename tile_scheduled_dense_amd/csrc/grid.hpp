// grid.hpp -- grids of many workgroups.  A dimension of a grid holds fewer than
// 2^32 threads: one of more is started cut to its low 32 bits, without an error.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tg {

// Whether `blocks` workgroups of `threads` fit one dimension.
inline bool grid_fits(int64_t blocks, int64_t threads) { return blocks < (int64_t(1) << 32) / threads; }

// Workgroups past kGridX lie in further rows of the grid, the last of which may
// reach past the work; wide_block is a workgroup's number.
constexpr int64_t kGridX = int64_t(1) << 22;
inline dim3 wide_grid(int64_t blocks) {
    return blocks <= kGridX ? dim3((unsigned)blocks) : dim3((unsigned)kGridX, (unsigned)((blocks + kGridX - 1) / kGridX));
}
__device__ __forceinline__ uint32_t wide_block() { return blockIdx.y * (uint32_t)kGridX + blockIdx.x; }

}  // namespace tg
