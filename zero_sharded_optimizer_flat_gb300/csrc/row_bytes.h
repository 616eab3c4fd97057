// How far a row of results goes.
#pragma once

#include <cuda_runtime.h>

namespace zopt {
namespace lm {

constexpr int kWarpCols = 128;  // at most: half a tile

// Bytes from column col to the end of a row of n columns of `size` bytes each, as far as a warp's part
// of a tile reaches; 0 or less where the row ends before col. (The whole row's may pass 31 bits.)
__host__ __device__ constexpr int row_bytes(int n, int col, int size) {
  return (n - col < kWarpCols ? n - col : kWarpCols) * size;
}

}  // namespace lm
}  // namespace zopt
