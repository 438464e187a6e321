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
// A thread has one block: 8 elements, loads and stores of 16 bytes, the loads
// under way while its numbers are drawn.  Bound: memory.  An element has 16 bits
// and not 32, so that the generator (18 products of 32 bits a block) stays
// below it with bf16 too.
#include "dropout.h"

#include <type_traits>

#include "grid_rows.h"
#include "prn_device.h"

namespace prn {
namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

__device__ __forceinline__ u32x4 philox(uint64_t block, uint64_t offset, uint64_t seed) {
  uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32);
  uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u, p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = xor3(static_cast<uint32_t>(p1 >> 32), c1, k0);
    c2 = xor3(static_cast<uint32_t>(p0 >> 32), c3, k1);
    c1 = static_cast<uint32_t>(p1);
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// Tensors from 128 MB on go past the caches, which hold 256 MB: 262144 x 512 bf16
// with a residual takes 125 us (6.4 TB/s), through them 135.  Smaller ones are
// often there already, or read next (a copy of 32 MB 10.7 us, past them 12.4).
constexpr int64_t kPastCaches = int64_t(1) << 27;

// eight values as memory has them
template <class T>
struct Eight {
  static constexpr int Q = sizeof(T) / 2;   // quads of 32 bits
  T v[8];
  template <bool PAST>
  __device__ __forceinline__ void load(const T* p) {
    u32x4 q[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const u32x4* const at = reinterpret_cast<const u32x4*>(p) + i;
      if constexpr (PAST) q[i] = __builtin_nontemporal_load(at); else q[i] = *at;
    }
    __builtin_memcpy(v, q, sizeof(v));
  }
  template <bool PAST>
  __device__ __forceinline__ void store(T* p) const {
    u32x4 q[Q];
    __builtin_memcpy(q, v, sizeof(v));
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      u32x4* const at = reinterpret_cast<u32x4*>(p) + i;
      if constexpr (PAST) __builtin_nontemporal_store(q[i], at); else *at = q[i];
    }
  }
};

// out may be x or residual: an element is read and written by one thread, which reads first
template <int DT, bool RES, bool PAST>
__global__ void __launch_bounds__(256) k_dropout(const typename Storage<DT>::T* x, const typename Storage<DT>::T* residual,
                                                 int64_t n, uint32_t drop, float scale, uint64_t seed, uint64_t offset,
                                                 const int64_t* __restrict__ state, typename Storage<DT>::T* out) {
  using ST = Storage<DT>;
  using E = Eight<typename ST::T>;
  const int64_t block = block_in_rows() * 256 + threadIdx.x, i0 = 8 * block, left = n - i0;
  if (left <= 0) return;
  if (state) {
    seed = static_cast<uint64_t>(state[0]);
    offset = static_cast<uint64_t>(state[1]);
  }
  auto finish = [&](const E& v, const E& r, E& o) {
    const u32x4 w = philox(static_cast<uint64_t>(block), offset, seed);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t number = e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu;
      const float y = number >= drop ? ST::load(&v.v[e]) * scale : 0.0f;   // a dropped NaN is dropped
      o.v[e] = ST::pack(RES ? y + ST::load(&r.v[e]) : y);
    }
  };
  E v = {}, r = {}, o;
  if (left >= 8) {
    v.template load<PAST>(x + i0);
    if constexpr (RES) r.template load<PAST>(residual + i0);
    finish(v, r, o);
    o.template store<PAST>(out + i0);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (e < left) v.v[e] = x[i0 + e];
    if (RES && e < left) r.v[e] = residual[i0 + e];
  }
  finish(v, r, o);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) out[i0 + e] = o.v[e];
}

}  // namespace

void launch_dropout(const DropoutArgs& a, const void* x, const void* residual, void* out) {
  const dim3 grid = rows_of_blocks((a.n + 2047) / 2048);
  auto go = [&](auto dt, auto res, auto past) {
    constexpr int DT = decltype(dt)::value;
    using T = typename Storage<DT>::T;
    k_dropout<DT, decltype(res)::value, decltype(past)::value><<<grid, 256, 0, a.stream>>>(
        static_cast<const T*>(x), static_cast<const T*>(residual), a.n, a.drop, a.scale, a.seed, a.offset, a.state,
        static_cast<T*>(out));
  };
  auto sized = [&](auto dt, auto res) {
    if (a.n * (a.bf16 ? 2 : 4) >= kPastCaches) go(dt, res, std::true_type{}); else go(dt, res, std::false_type{});
  };
  auto typed = [&](auto res) {
    if (a.bf16) sized(std::integral_constant<int, kBF16>{}, res); else sized(std::integral_constant<int, kF32>{}, res);
  };
  if (residual) typed(std::true_type{}); else typed(std::false_type{});
}

}  // namespace prn
