// Launches of more workgroups than one dimension of a grid may have.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace prn {

// A launch has fewer than 2^32 threads along x: more workgroups than fit go in
// rows of 2^21 along y, the last row with some to spare.
inline dim3 rows_of_blocks(int64_t n, int64_t z = 1) {
  constexpr int64_t kRow = int64_t(1) << 21;
  return n <= kRow ? dim3(unsigned(n), 1, unsigned(z)) : dim3(unsigned(kRow), unsigned((n + kRow - 1) / kRow), unsigned(z));
}
__device__ __forceinline__ int64_t block_in_rows() { return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x; }

}  // namespace prn
