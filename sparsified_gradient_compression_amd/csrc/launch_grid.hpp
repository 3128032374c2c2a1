// launch_grid.hpp -- grids of any number of workgroups.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace dgc {

// A launch may have fewer than 2^32 threads along x.  More workgroups lie in
// rows of so many along y: a multiple of 8, so that a workgroup's number
// modulo 8 still names its die.
constexpr int64_t kGridRow = int64_t(1) << 20;

// At least `blocks` (up to 2^31 - 1) workgroups of `threads` (up to 1024) each.
inline dim3 grid_of(int64_t blocks, int threads) {
    if (blocks * threads < int64_t(1) << 32) return dim3(static_cast<unsigned>(blocks));
    return dim3(static_cast<unsigned>(kGridRow),
                static_cast<unsigned>((blocks + kGridRow - 1) / kGridRow));
}

// The workgroup's number in such a grid.  The last row may go beyond `blocks`.
__device__ __forceinline__ int64_t block_number() {
    return int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
}

}  // namespace dgc
