// How the tiles of a large product are dealt to the device, for the vocabulary
// loss and the feed-forward product: tiles of 256 x 256 or 256 x 192
// (mm_tile.h), one workgroup a CU.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace prn {

constexpr int kXcd = 8;
constexpr int64_t kCus = 256;
constexpr int64_t kTileRows = 256, kTileCols = 256;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Workgroups are dealt round-robin to the XCDs.  The units of work of this
// workgroup, when every XCD takes a contiguous share of them, in proportion
// to its workgroups, so that neighbouring units share its L2.
struct Units {
  uint32_t u, step, end;
  __device__ __forceinline__ explicit Units(uint32_t units) {
    const uint32_t grid = gridDim.x, x = blockIdx.x % kXcd, slot = blockIdx.x / kXcd;
    const uint32_t q = grid / kXcd, rem = grid % kXcd, before = x * q + min(x, rem);
    step = q + (x < rem ? 1 : 0);
    u = static_cast<uint32_t>(static_cast<uint64_t>(units) * before / grid) + slot;
    end = static_cast<uint32_t>(static_cast<uint64_t>(units) * (before + step) / grid);
  }
  __device__ __forceinline__ bool valid() const { return u < end; }
  __device__ __forceinline__ void advance() { u += step; }
};
// tile u of rows x cols in groups of `group` rows, walked down the group's rows first
__device__ __forceinline__ void tile_of(uint32_t u, uint32_t rows, uint32_t cols, uint32_t group, uint32_t& r, uint32_t& c) {
  const uint32_t per = group * cols, g = u / per, in = u - g * per;
  const uint32_t h = min(group, rows - g * group);
  c = in / h;
  r = g * group + in - c * h;
}

// A product's work: the rows whose tiles fill whole rounds of the device run
// over the whole sum each; the sum of the rest is cut in slices, joined after.
// The fewest microseconds of a few slice counts, with and without a head.
struct Cut {
  int64_t head;       // rows of the first kind
  int64_t s, len;     // slices of the rest's sum, and their length
};
inline Cut cut_of(int64_t rows, int64_t K, int64_t d, int terms, int64_t bn, double* us) {
  // microseconds of a CU for a tile over k of the sum (256 x 256 at 1.05
  // PFLOP/s of the device), and of storing fp32 sums and reading them again at
  // 4 TB/s, weighed half as much again: CUs that idle in a round leave the others
  // their power (16384 x 520 x 16384 with dx's 192 tiles in four slices of the
  // sum took 1093 us, in one 1066; 5003 x 520 x 50021 without the rest's slices
  // 1056, with them 1016)
  auto tile = [&](int64_t k) { return double(k) * terms * kTileRows * bn * (bn == kTileCols ? 1.0 : 1.12) * 2 / 4.1e6; };
  auto join = [&](int64_t n, int64_t s) { return s > 1 ? 4 + double(s) * n * d * 8 * 1.5 / 4e6 : 0.0; };
  const int64_t n_col = cdiv(d, bn), blocks = cdiv(rows, kTileRows), whole = blocks * n_col / kCus * kCus;
  Cut best{};
  *us = -1;
  for (int64_t head = 0;; head = std::min(whole / n_col * kTileRows, rows)) {
    const int64_t rest = rows - head, tiles = cdiv(rest, kTileRows) * n_col;
    const double first = cdiv(cdiv(head, kTileRows) * n_col, kCus) * tile(K) + (head > 0 && rest > 0 ? 3 : 0);
    for (int64_t want : {int64_t(1), int64_t(2), int64_t(3), int64_t(4), int64_t(6), int64_t(8), tiles ? std::min(kCus / tiles, K / 512) : 1}) {
      if (want < 1 || (want > 1 && K / want < 512)) continue;
      const int64_t len = cdiv(cdiv(K, want), 64) * 64, n = cdiv(K, len);
      const double t = first + cdiv(tiles * n, kCus) * tile(len) + join(rest, n);
      if (*us < 0 || t < *us) {
        *us = t;
        best = {head, n, len};
      }
    }
    if (head > 0 || whole / n_col == 0) break;
  }
  return best;
}

}  // namespace prn
