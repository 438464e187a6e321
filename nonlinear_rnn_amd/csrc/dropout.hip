// Dropout from a counter, whose mask is never stored.
//
//   out = residual + (kept ? x scale : 0)        kept: number of the element >= drop
//
// The numbers are 16 bits each, eight of them from one block of Philox4x32-10
// (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", 2011): key the seed, counter (index / 8, offset), both 64 bits.
// Element 8 b + 2 j has the low half of word j of block b, 8 b + 2 j + 1 the
// high half.  So the mask is a function of (seed, offset, index) alone, the
// same in both directions, for every type, shape and launch.
//
// A thread has one block: 8 elements, loads and stores of 16 bytes.  Bound: in
// fp32 memory, in bf16 memory and the generator's 20 products of 32 bits a
// block about alike, which is why an element has 16 bits and not 32.
#include "dropout.h"

#include <type_traits>

#include "grid_rows.h"
#include "prn_device.h"

namespace prn {
namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

__device__ __forceinline__ u32x4 philox(uint64_t block, uint64_t offset, uint64_t seed) {
  uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32);
  uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u, p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(p1);
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

template <int DT>
__global__ void __launch_bounds__(256) k_dropout(const typename Storage<DT>::T* __restrict__ x,
                                                 const typename Storage<DT>::T* __restrict__ residual, int64_t n,
                                                 uint32_t drop, float scale, uint64_t seed, uint64_t offset,
                                                 const int64_t* __restrict__ state, typename Storage<DT>::T* __restrict__ out) {
  using ST = Storage<DT>;
  const int64_t block = block_in_rows() * 256 + threadIdx.x, i0 = 8 * block;
  if (i0 >= n) return;
  if (state) {
    seed = static_cast<uint64_t>(state[0]);
    offset = static_cast<uint64_t>(state[1]);
  }
  typename ST::T v[8], r[8], o[8];
  const bool whole = i0 + 8 <= n;
  if (whole) {
    __builtin_memcpy(v, __builtin_assume_aligned(x + i0, 16), sizeof(v));
    if (residual) __builtin_memcpy(r, __builtin_assume_aligned(residual + i0, 16), sizeof(r));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = i0 + e < n ? x[i0 + e] : typename ST::T(0);
      r[e] = residual && i0 + e < n ? residual[i0 + e] : typename ST::T(0);
    }
  }
  const u32x4 w = philox(static_cast<uint64_t>(block), offset, seed);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t number = e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu;
    float y = number >= drop ? ST::load(&v[e]) * scale : 0.0f;   // a dropped NaN is dropped
    if (residual) y += ST::load(&r[e]);
    o[e] = ST::pack(y);
  }
  if (whole) {
    __builtin_memcpy(__builtin_assume_aligned(out + i0, 16), o, sizeof(o));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i0 + e < n) out[i0 + e] = o[e];
  }
}

}  // namespace

void launch_dropout(const DropoutArgs& a, const void* x, const void* residual, void* out) {
  const dim3 grid = rows_of_blocks((a.n + 2047) / 2048);
  auto go = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    using T = typename Storage<DT>::T;
    k_dropout<DT><<<grid, 256, 0, a.stream>>>(static_cast<const T*>(x), static_cast<const T*>(residual), a.n, a.drop, a.scale,
                                              a.seed, a.offset, a.state, static_cast<T*>(out));
  };
  if (a.bf16) go(std::integral_constant<int, kBF16>{}); else go(std::integral_constant<int, kF32>{});
}

}  // namespace prn
