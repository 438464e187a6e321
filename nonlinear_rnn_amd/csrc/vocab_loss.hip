// Softmax cross entropy over a vocabulary, and its gradients, without the
// N x V logits in memory.
//
//   z = s x W^T          lse_n = log sum_v exp z_nv     loss_n = lse_n - z_n,t(n)
//   dz_nv = s ((dloss_n + dlse_n) p_nv - dloss_n [v = t(n)])     p = exp(z - lse)
//   dx = dz W            dW = dz^T x
//
// Forward: a workgroup keeps a tile of tokens and walks a range of the
// vocabulary; every tile of logits stays in the matrix-core accumulators
// and is folded into a running maximum and sum of the lane's token (the
// tile is W rows x tokens, so that a lane holds one token and many vocabulary
// entries).  The ranges' (maximum, sum) pairs are joined per token.
// Backward, in pieces of the vocabulary: the tile of logits is formed again,
// turned into dz and stored (fp16; fp32 data: as two fp16 terms); then
// dx += dz W and dW = dz^T x of the piece.  8 N V d operations in all, two of
// them for the logits' second time.
//
// The matrix cores take 16-bit operands.
// bf16 data: the forward's logits are products of the values as they are.  dz
// is rounded to fp16, not bf16: an entry is then off by 2^-11 of itself at
// most, not 2^-8 (the entry of the target can carry the whole row); bf16 took
// the error of dx and dW, 0.0017 from their own rounding, to 0.0019.  W and x
// are laid out as fp16 for the backward's products, which holds bf16's eight
// bits exactly (down to 2^-31 of the largest value, below that to 2^-39 of it).
// fp32 data: x, W and dz run as two fp16 terms, v = hi + lo to 2^-22 |v|, three
// products each (lo lo, below 2^-22, is left out).  That is four fp32
// roundings a product, below what the fp32 sums over them make; the exact
// three-term bf16 split (bf16split.h) took twice the products and 1.74 ms
// where this takes 0.86 (4096 x 256 x 32000).
// For fp16's range W is scaled by the power of two that takes its largest value
// to 2^14 .. 2^15, every token's x by that of its own (so that a large token
// leaves the others' logits alone), and every token's row of dz, in units of its
// weight, the power of two below the larger of |dloss| and |dloss + dlse|, by
// 2^13 (so that a light token's row of dx is as good as a heavy one's).  dW, which
// sums over tokens, takes x times the weight, scaled by the power of two of the
// largest of these.  A W of values far apart (kNear) has a unit for each larger
// row in the logits and for each column in dx, so that a channel of mask values
// leaves the other entries and channels alone.  Values below 2^-17 of the largest
// one lose the low bits of lo: at most 2^-39 of the largest, half a step of 2^-24
// over 2^14; an entry of dz is off by at most 2^-38 of its token's weight, half a
// step of 2^-24 over 2^13, however small it is.  The units come back, in fp32,
// where they are used.  Everything is summed in fp32 in a fixed order.
#include "vocab_loss.h"

#include <algorithm>
#include <type_traits>

#include "grid_rows.h"
#include "mm_tile.h"
#include "prn_device.h"

namespace prn {
namespace {

constexpr int kTerms = 3;   // products of two-term operands

// 8 waves, 256 x 256, 128 KB: the least traffic per product; one workgroup a CU
template <bool PAIR> using Big = MmTile<2, 4, 4, 2, 64, 2, PAIR>;
// 256 x 128 for the logits of few tokens: bf16 data 4 waves, 72 KB, two
// workgroups a CU; fp32 data 8 waves, 96 KB
template <bool PAIR>
using Mid = std::conditional_t<PAIR, MmTile<4, 2, 2, 2, 64, 2, true>, MmTile<2, 2, 4, 2, 32, 3, false>>;
// 8 waves, 256 x 192, 112 KB: for dx and dW where 256 columns a tile would be wider than the rows
template <bool PAIR> using Wide = MmTile<4, 2, 2, 3, 64, 2, PAIR>;
// few tokens: 128 x 64
template <bool PAIR> using Few = MmTile<4, 1, 1, 2, 64, 3, PAIR>;
// tiles' extents, and workgroups of Mid on a CU
constexpr int64_t kBM = Big<false>::BM, kBig = Big<false>::BN, kMid = Mid<false>::BN, kWide = Wide<false>::BN;
constexpr int64_t kFewM = Few<false>::BM, kFewN = Few<false>::BN;
int64_t mid_slots(bool bf16) { return bf16 ? 2 : 1; }
constexpr int kXcd = 8;

// A factor of the logits, above 0 also where their operands' units are so small
// that it underflows: an entry past the vocabulary is -inf times it, and the
// logits, below 2^60 in these units, are zero all the same.
__device__ __forceinline__ float above_zero(float c) { return fmaxf(c, 0x1p-126f); }

// Exponents (of 2) of this size and more are formed as the factor times a
// difference: the fused product less the rounded other one, an instruction
// shorter, is off by 2^-12 there, and by whole powers of 2 at logits of 1e7.
constexpr float kFar = 0x1p12f;

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

// ------------------------------------------------------------ operands ---

// A copy of bf16 rows of d values as rows of ldp, zeros past d.  One thread
// per 8 columns.
__global__ void __launch_bounds__(256) k_loss_pad(const uint16_t* __restrict__ in, int64_t R, int64_t d, int64_t ldp,
                                                  uint16_t* __restrict__ out) {
  const int64_t C = ldp / 8;
  const int64_t i = block_in_rows() * 256 + threadIdx.x;
  if (i >= R * C) return;
  const int64_t r = i / C;
  const int c0 = static_cast<int>(i - r * C) * 8;
  mm_s16x8 v;
  if (c0 + 8 <= d) {   // one load, aligned or not
    __builtin_memcpy(&v, in + r * d + c0, sizeof(v));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c0 + e < d ? static_cast<short>(in[r * d + c0 + e]) : short(0);
  }
  *reinterpret_cast<mm_s16x8*>(out + r * ldp + c0) = v;
}

constexpr int kMaxParts = 1024;
constexpr int kUnit = 13;   // dz is stored times 2^13: fp16 has entries down to 2^-37

constexpr float kNoExponent = -1e4f;   // of nothing but zeros
// W has one unit where every eight neighbouring values have one within 2^kNear
// of the largest (or none but zeros).  Where not, rows of up to 2^kNear times the
// smallest of those share one, and each larger row (with a mask's value among its
// channels, say) has its own in the logits, and every column in dx: the gradients
// of 32768 x 512 x 32768, 5003 x 520 x 50021 and 4096 x 256 x 32000 (fp32) with
// eight channels of W a millionth take 3670, 1087 and 721 us against 3512, 993 and
// 686.
constexpr float kNear = 12.0f;

// The units of a call
struct LossUnits {
  float iw;                        // z = acc iw s times the token's inverse unit (and the row's, row_unit)
  int32_t exponent;                // W's common one
  int32_t wide;                    // has it others?
  int32_t shift;                   // xg = u x 2^shift
  int32_t odd;                     // has a row its own, or is a token's lse2 kFar or more? (RowFar)
  float parts[3][kMaxParts];       // the workgroups' maxima: of the exponents of u x; of W's eights' and their negatives
};

template <class T>
__device__ __forceinline__ int64_t target_at(const void* targets, int64_t n) {
  return static_cast<int64_t>(static_cast<const T*>(targets)[n]);
}
__device__ __forceinline__ int64_t target_of(const void* targets, int bytes, int64_t n) {
  return bytes == 4 ? target_at<int32_t>(targets, n) : target_at<int64_t>(targets, n);
}

__device__ __forceinline__ float block_max(float m, float* w) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = m;
  __syncthreads();
  for (int i = 0; i < static_cast<int>(blockDim.x >> 6); ++i) m = fmaxf(m, w[i]);
  return m;
}
__device__ __forceinline__ float join_parts(const float* part, int parts, float* w) {
  float m = kNoExponent;
  for (int q = threadIdx.x; q < parts; q += blockDim.x) m = fmaxf(m, part[q]);
  return block_max(m, w);
}
__device__ __forceinline__ float two_to(int e) { return ldexpf(1.0f, e); }
__device__ __forceinline__ float finite_max(float m, float v) {
  v = fabsf(v);
  return v < __builtin_inff() ? fmaxf(m, v) : m;
}

__device__ __forceinline__ int exponent_of(float m) { return max(static_cast<int>(__float_as_uint(m) >> 23) - 127, -126); }

// What arrives at a token's loss and at its lse and loss together, and its
// weight u: the power of two below the larger one (0: neither, or not finite).
// Its row of dz is stored as 2^kUnit dz / (s u), so that every token's row of
// dx is as good as it would be alone.
struct Arriving {
  float one, both, u;
};
__device__ __forceinline__ Arriving arriving(const float* dloss, const float* dlse, int64_t n, bool ignored) {
  Arriving a;
  a.one = ignored ? 0.0f : dloss[n];
  a.both = dlse ? a.one + dlse[n] : a.one;
  const float m = finite_max(finite_max(0.0f, a.one), a.both);
  a.u = m > 0.0f ? __uint_as_float(static_cast<uint32_t>(exponent_of(m) + 127) << 23) : 0.0f;
  return a;
}

// eight values of each of M rows (row(q) the q-th) from column c0 on, zeros past d
template <bool BF16, int M, class Row>
__device__ __forceinline__ void raw8(const void* p, Row row, int64_t d, int64_t c0,
                                     typename Storage<BF16 ? kBF16 : kF32>::T (&t)[M][8]) {
  using T = typename Storage<BF16 ? kBF16 : kF32>::T;
  const T* const at = static_cast<const T*>(p) + c0;
  if (c0 + 8 <= d) {   // at once, aligned or not
#pragma unroll
    for (int q = 0; q < M; ++q) __builtin_memcpy(t[q], at + row(q) * d, sizeof(t[q]));
  } else {
#pragma unroll
    for (int q = 0; q < M; ++q)
#pragma unroll
      for (int e = 0; e < 8; ++e) t[q][e] = c0 + e < d ? at[row(q) * d + e] : T(0);
  }
}

// The largest finite magnitudes of rows r, r + step, .. of R in all, `lanes` lanes
// a row and two rows in flight (four take registers of which the occupancy
// suffers): take(row, magnitude), in every lane.
template <bool BF16, class Take>
__device__ __forceinline__ void row_maxima(const void* p, int64_t r, int64_t step, int64_t R, int64_t d, int lanes, Take take) {
  constexpr int kRows = 2;
  const int lane = threadIdx.x % lanes;
  for (; r < R; r += kRows * step) {
    float m[kRows] = {};
    for (int64_t c0 = 8 * lane; c0 < d; c0 += 8 * lanes) {
      typename Storage<BF16 ? kBF16 : kF32>::T t[kRows][8];
      raw8<BF16>(p, [&](int q) { return imin(r + q * step, R - 1); }, d, c0, t);
#pragma unroll
      for (int q = 0; q < kRows; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) m[q] = finite_max(m[q], Storage<BF16 ? kBF16 : kF32>::load(&t[q][e]));
    }
    for (int o = 1; o < lanes; o <<= 1) {
#pragma unroll
      for (int q = 0; q < kRows; ++q) m[q] = fmaxf(m[q], __shfl_xor(m[q], o, 64));
    }
#pragma unroll
    for (int q = 0; q < kRows; ++q)
      if (r + q * step < R) take(r + q * step, m[q]);
  }
}

// Workgroups [0, n1): the tokens' largest magnitudes, `lanes` lanes a token, to
// top_x, and the greatest of the exponents of u x (for dW, where there is a
// dloss).  The last n2: the greatest and the least exponent of W's eights.  Values
// that are not finite do not set a unit, they go through as they are.
template <bool BF16>
__global__ void __launch_bounds__(256) k_loss_maxima(const float* __restrict__ dloss, const float* __restrict__ dlse,
                                                     const void* __restrict__ targets, int target_bytes, int64_t ignore,
                                                     int64_t N, int64_t V, int64_t d, int64_t ldp, const void* __restrict__ x,
                                                     const void* __restrict__ W, int n1, int lanes, int n2,
                                                     LossUnits* __restrict__ u, float* __restrict__ top_x,
                                                     uint32_t* __restrict__ columns) {
  using S = Storage<BF16 ? kBF16 : kF32>;
  __shared__ float w[4];
  int b = static_cast<int>(blockIdx.x);
  const int per = 256 / lanes;
  const bool first = threadIdx.x % lanes == 0;
  if (b == 0) {
    if (columns)
      for (int64_t c = threadIdx.x; c < ldp; c += 256) columns[c] = 0;
  }
  float top = kNoExponent, low = kNoExponent;
  if (b < n1) {
    row_maxima<BF16>(x, static_cast<int64_t>(b) * per + threadIdx.x / lanes, static_cast<int64_t>(n1) * per, N, d, lanes,
                     [&](int64_t n, float m) {
                       if (!first) return;
                       top_x[n] = m;
                       if (!dloss) return;
                       const Arriving a = arriving(dloss, dlse, n, target_of(targets, target_bytes, n) == ignore);
                       if (m > 0.0f && a.u > 0.0f) top = fmaxf(top, static_cast<float>(exponent_of(m) + exponent_of(a.u)));
                     });
    top = block_max(top, w);
    if (threadIdx.x == 0) u->parts[0][b] = top;
    return;
  }
  b -= n1;
  const int64_t n = V * d;
#pragma unroll 4
  for (int64_t i = (static_cast<int64_t>(b) * 256 + threadIdx.x) * 8; i < n; i += static_cast<int64_t>(n2) * 2048) {
    typename S::T t[8];
    const typename S::T* const q = static_cast<const typename S::T*>(W) + i;
    if (i + 8 <= n) {
      __builtin_memcpy(t, __builtin_assume_aligned(q, 16), sizeof(t));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = i + e < n ? q[e] : typename S::T(0);
    }
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = finite_max(m, S::load(&t[e]));
    if (m > 0.0f) {
      top = fmaxf(top, static_cast<float>(exponent_of(m)));
      low = fmaxf(low, -static_cast<float>(exponent_of(m)));
    }
  }
  top = block_max(top, w);
  low = block_max(low, w);
  if (threadIdx.x == 0) {
    u->parts[1][b] = top;
    u->parts[2][b] = low;
  }
}

// Joins the maxima and writes the units (the first workgroup); of a W of more than
// one unit, workgroups [0, n1) the rows' largest magnitudes, to top_w, the others
// the columns', as bits (so that it does not matter in which order they meet): 256
// columns each, 8 a lane, 32 rows at a time of its share.
template <bool BF16>
__global__ void __launch_bounds__(1024) k_loss_units(const void* __restrict__ W, int64_t V, int64_t d, int n1, int lanes,
                                                     int blocks, int64_t share, LossUnits* __restrict__ u, int parts1,
                                                     int parts2, int gradients, float* __restrict__ top_w,
                                                     uint32_t* __restrict__ top) {
  constexpr int kRows = 4;
  __shared__ float w[16];
  __shared__ float hand[32][256];
  const float greatest = join_parts(u->parts[1], parts2, w), least = -join_parts(u->parts[2], parts2, w);
  const bool wide = greatest > kNoExponent && greatest > least + kNear;
  if (blockIdx.x == 0) {
    const float most = gradients ? join_parts(u->parts[0], parts1, w) : kNoExponent;
    if (threadIdx.x == 0) {
      u->exponent = greatest > kNoExponent ? static_cast<int>(fmaxf(fminf(greatest, least + kNear), -112.0f)) : 14;
      u->iw = two_to(u->exponent - 14);
      u->wide = wide;
      u->shift = most > kNoExponent ? 14 - static_cast<int>(most) : 0;
      u->odd = 0;
    }
  }
  if (!wide) return;
  const int tid = threadIdx.x, b = static_cast<int>(blockIdx.x);
  if (b < n1) {
    const int per = 1024 / lanes;
    row_maxima<BF16>(W, static_cast<int64_t>(b) * per + tid / lanes, static_cast<int64_t>(n1) * per, V, d, lanes,
                     [&](int64_t r, float m) {
                       if (tid % lanes == 0) top_w[r] = m;
                     });
    return;
  }
  const int lane = tid & 31, g = tid >> 5;
  const int64_t first = static_cast<int64_t>((b - n1) % blocks) * 256, c0 = first + 8 * lane;
  const int64_t r0 = static_cast<int64_t>((b - n1) / blocks) * share, r1 = imin(r0 + share, V);
  float m[8] = {};
  if (c0 < d) {
    for (int64_t r = r0 + g; r < r1; r += 32 * kRows) {
      typename Storage<BF16 ? kBF16 : kF32>::T t[kRows][8];
      raw8<BF16>(W, [&](int q) { return imin(r + 32 * q, r1 - 1); }, d, c0, t);
#pragma unroll
      for (int q = 0; q < kRows; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) m[e] = finite_max(m[e], Storage<BF16 ? kBF16 : kF32>::load(&t[q][e]));
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) hand[g][8 * lane + e] = m[e];
  __syncthreads();
  if (tid >= 256 || first + tid >= d) return;
  float t = hand[0][tid];
#pragma unroll 8
  for (int q = 1; q < 32; ++q) t = fmaxf(t, hand[q][tid]);
  atomicMax(top + first + tid, __float_as_uint(t));
}

// the power of two that takes a largest value m to 2^14 .. 2^15 (a token's of its
// x), and its inverse
__device__ __forceinline__ float unit_of(float m, float* inverse) {
  const int e = m > 0.0f ? static_cast<int>(__float_as_uint(m) >> 23) - 127 : 14;
  const int k = min(max(14 - e, -126), 126);
  *inverse = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
}

__device__ __forceinline__ float inverse_unit(float m) {
  float inverse;
  unit_of(m, &inverse);
  return inverse;
}

// A token's row of dz in its units: sign 2^(|c| acc - lse2) - one at the target.
// The magnitude of (dloss + dlse) / u is folded into the exponent.
struct RowCoef {
  float c;              // s log2(e) times the units of its logits; the sign is that of (dloss + dlse)
  float one, lse2;
  int32_t target;       // -1: none
};

// The same for a token whose lse2 is kFar and more, where it holds little of a
// fraction: sign 2^((acc back - lse) log2(e) + log2p).  acc back - lse, both as
// the forward had them, is at most what lse's rounding makes it.
struct RowFar {
  float back, lse, log2p, unused;
};
__device__ __forceinline__ bool is_far(float lse2) { return fabsf(lse2) >= kFar && fabsf(lse2) < __builtin_inff(); }

// eight values' fp16 terms, to row r from column c0 on
template <bool BF16>
__device__ __forceinline__ void store_terms(const float* v, uint16_t* to, int64_t r, int64_t ldp, int64_t c0) {
  mm_f16x8 hi, lo;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    hi[e] = static_cast<_Float16>(v[e]);
    lo[e] = static_cast<_Float16>(v[e] - static_cast<float>(hi[e]));
  }
  if constexpr (BF16) {
    *reinterpret_cast<mm_f16x8*>(to + r * ldp + c0) = hi;
  } else {
    uint16_t* const out = to + 2 * (r * ldp + (c0 & ~int64_t(31))) + (c0 & 31);
    *reinterpret_cast<mm_f16x8*>(out) = hi;
    *reinterpret_cast<mm_f16x8*>(out + 32) = lo;
  }
}

// Lays out x and W in fp16 terms, rows of ldp values (fp32 data: 2 ldp, every
// 32 high terms and their 32 low ones), zeros past d, 8 columns a thread.
// Workgroups [0, n1): x, to xh in units of the token, and for the gradients to xg,
// for dW, times the token's weight u and in units of the largest of these; u and
// the token's coefficients.  The others W, to wh in W's unit, or the row's own
// (what that is larger to row_unit), and, where it has more than one, for dx to wd
// in units of the column.
template <bool BF16>
__global__ void __launch_bounds__(256) k_loss_layout(const float* __restrict__ dloss, const float* __restrict__ dlse,
                                                     const float* __restrict__ lse, const void* __restrict__ targets,
                                                     int target_bytes, int64_t ignore, int64_t N, int64_t V, int64_t d,
                                                     float scale, int64_t ldp, const void* __restrict__ x,
                                                     const void* __restrict__ W, int n1, LossUnits* __restrict__ units, const float* __restrict__ top_x,
                                                     const float* __restrict__ top_w, float* __restrict__ row_unit,
                                                     const uint32_t* __restrict__ columns, float* __restrict__ weight,
                                                     RowCoef* __restrict__ coef, RowFar* __restrict__ far,
                                                     uint16_t* __restrict__ xh, uint16_t* __restrict__ xg,
                                                     uint16_t* __restrict__ wh, uint16_t* __restrict__ wd) {
  using S = Storage<BF16 ? kBF16 : kF32>;
  const int64_t b = block_in_rows();
  const bool is_x = b < n1;
  const int64_t R = is_x ? N : V, C = ldp / 8, i = (is_x ? b : b - n1) * 256 + threadIdx.x;
  if (i >= R * C) return;
  const int64_t r = i / C, c0 = (i - r * C) * 8;
  typename S::T t[1][8];
  raw8<BF16>(is_x ? x : W, [&](int) { return r; }, d, c0, t);
  float v[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = S::load(&t[0][e]);
  if (!is_x) {
    const bool wide = units->wide != 0;
    int own = units->exponent;
    if (wide) own = max(exponent_of(top_w[r]), own);   // (zeros: the common one)
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = ldexpf(v[e], 14 - own);
    store_terms<BF16>(s, wh, r, ldp, c0);
    if (wd && wide) {
      uint32_t k[8];
      __builtin_memcpy(k, __builtin_assume_aligned(columns + c0, 32), sizeof(k));
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = ldexpf(v[e], 14 - exponent_of(__uint_as_float(k[e])));
      store_terms<BF16>(s, wd, r, ldp, c0);
    }
    if (c0 == 0) {
      row_unit[r] = two_to(min(own - units->exponent, 127));
      if (own > units->exponent) units->odd = 1;
    }
    return;
  }
  float inverse;
  const float unit = unit_of(top_x[r], &inverse);
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = v[e] * unit;
  store_terms<BF16>(s, xh, r, ldp, c0);
  if (!xg) return;
  const int64_t target = target_of(targets, target_bytes, r);
  const Arriving in = arriving(dloss, dlse, r, target == ignore);
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = in.u > 0.0f ? ldexpf(v[e], units->shift + exponent_of(in.u)) : v[e] * 0.0f;
  store_terms<BF16>(s, xg, r, ldp, c0);
  if (c0 != 0) return;
  weight[r] = in.u;
  const float u = in.u > 0.0f ? in.u : 1.0f, p = in.both / u;
  const float iw = units->iw;
  RowCoef k;
  k.c = copysignf(above_zero(scale * kLog2e * iw * inverse), p);
  k.one = in.one / u * (1 << kUnit);
  // no such entry: the loss was NaN, and so is its gradient
  const bool lost = target != ignore && (target < 0 || target >= V);
  const float log2p = log2f(fabsf(p)), l = lse[r];
  k.lse2 = lost ? __builtin_nanf("") : fmaf(l, kLog2e, -log2p) - kUnit;   // p = 0: +inf, a row of zeros
  k.target = target == ignore || lost ? -1 : static_cast<int32_t>(target);
  coef[r] = k;
  far[r] = {iw * inverse * scale, l, log2p + kUnit, 0.0f};
  if (is_far(k.lse2)) units->odd = 1;
}

// ------------------------------------------------------------- forward ---

// part[n][split] = (maximum, sum of 2^(c (z - maximum))) of token n over the
// split's vocabulary tiles, z the plain products x W^T (F16: of the operands
// in their units), c = s log2(e) > 0 (F16: in those units, the token's own).
// A unit is a token tile and a split; four token tiles and their splits are
// neighbours, so that an XCD's workgroups share the W tiles they walk (8 or 16
// were 1 to 5% slower).
template <class Tl, bool F16>
__global__ void __launch_bounds__(Tl::NTHR, 2) k_loss_lse(MmOperand W, MmOperand X, int64_t N, int64_t V, int64_t d,
                                                          float c_, const LossUnits* __restrict__ units,
                                                          const float* __restrict__ top_x,
                                                          const float* __restrict__ row_unit, int n_tok, int splits,
                                                          int per_split, float2* __restrict__ part) {
  if constexpr (F16) c_ *= units->iw;
  const bool odd = F16 && __builtin_amdgcn_readfirstlane(units->odd) != 0;
  auto factor = [&](int64_t n) { return F16 ? above_zero(c_ * inverse_unit(top_x[imin(n, N - 1)])) : c_; };
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Tl::LDS];
  __shared__ float2 hand[Tl::WR][Tl::BN];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, l32 = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / Tl::WC, wc = wave % Tl::WC;
  const uint32_t v_tiles = static_cast<uint32_t>((V + Tl::BM - 1) / Tl::BM);
  Tl tile;
  tile.open(lds, W, V, X, N, 0, d);
  // the loads' place: unit, vocabulary tile
  Units lu(static_cast<uint32_t>(n_tok) * splits), cu(lu);
  uint32_t lt = 0, lt1 = 0, ltok = 0;
  auto enter = [&]() {
    if (!lu.valid()) return false;
    uint32_t split;
    tile_of(lu.u, n_tok, splits, 4, ltok, split);
    lt = split * per_split;
    lt1 = min(lt + per_split, v_tiles);
    return true;
  };
  auto next = [&]() {
    if (++lt == lt1) {
      lu.advance();
      if (!enter()) return;
    }
    tile.template seek<false, false>(static_cast<int64_t>(lt) * Tl::BM, static_cast<int64_t>(ltok) * Tl::BN);
  };
  if (!enter()) return;
  tile.template seek<false, false>(static_cast<int64_t>(lt) * Tl::BM, static_cast<int64_t>(ltok) * Tl::BN);
  tile.template prime<false, false>(next);
  for (; cu.valid(); cu.advance()) {
    uint32_t tok, split;
    tile_of(cu.u, n_tok, splits, 4, tok, split);
    const int64_t n0 = static_cast<int64_t>(tok) * Tl::BN;
    const uint32_t t0 = split * per_split, t1 = min(t0 + per_split, v_tiles);
    // a lane's sums are taken against the maximum m of the first tile that
    // had one; a later maximum replaces it only when the sums grow large
    float m[Tl::WN], s[Tl::WN], c[Tl::WN];
#pragma unroll
    for (int j = 0; j < Tl::WN; ++j) {
      m[j] = s[j] = 0.0f;
      c[j] = factor(n0 + (wc * Tl::WN + j) * 32 + l32);
    }
    for (uint32_t t = t0; t < t1; ++t) {
      const int64_t v0 = static_cast<int64_t>(t) * Tl::BM;
      tile.template multiply<false, false, false, F16>(next);
      if constexpr (F16) {
        if (odd) {   // rows of W in units of their own
#pragma unroll
          for (int i = 0; i < Tl::WM; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 f = *reinterpret_cast<const float4*>(row_unit + v0 + (wr * Tl::WM + i) * 32 + 8 * q + 4 * half);
#pragma unroll
              for (int j = 0; j < Tl::WN; ++j) {
                tile.acc[i][j][4 * q] *= f.x;
                tile.acc[i][j][4 * q + 1] *= f.y;
                tile.acc[i][j][4 * q + 2] *= f.z;
                tile.acc[i][j][4 * q + 3] *= f.w;
              }
            }
        }
      }
      if (v0 + Tl::BM > V) {
        const int left = static_cast<int>(V - v0) - wr * Tl::WM * 32 - 4 * half;
#pragma unroll
        for (int i = 0; i < Tl::WM; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
#pragma unroll
            for (int j = 0; j < Tl::WN; ++j)
              tile.acc[i][j][r] = 32 * i + 8 * (r >> 2) + (r & 3) < left ? tile.acc[i][j][r] : -__builtin_inff();
      }
#pragma unroll
      for (int j = 0; j < Tl::WN; ++j) {
        auto sum_against = [&](float ref) {
          float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          const float off = -ref * c[j];
          const bool far = fabsf(off) >= kFar;
          if (__builtin_amdgcn_ballot_w64(far)) {
            asm volatile("");   // a branch, for some lane's token; the others' exponents are as without it
#pragma unroll
            for (int i = 0; i < Tl::WM; ++i)
#pragma unroll
              for (int r = 0; r < 16; ++r) {
                const float a = tile.acc[i][j][r];
                q[r & 3] += ex2(far ? (a - ref) * c[j] : fmaf(a, c[j], off));
              }
          } else {
#pragma unroll
            for (int i = 0; i < Tl::WM; ++i)
#pragma unroll
              for (int r = 0; r < 16; ++r) q[r & 3] += ex2(fmaf(tile.acc[i][j][r], c[j], off));
          }
          return (q[0] + q[1]) + (q[2] + q[3]);
        };
        float sum = sum_against(m[j]);
        // no maximum yet, or this tile's sum is out of proportion (or NaN)
        const bool renew = s[j] == 0.0f || !(sum < 0x1p60f);
        if (__builtin_amdgcn_ballot_w64(renew)) {
          asm volatile("");   // a branch: taken once or twice a unit; for these lanes only
          float mx = tile.acc[0][j][0];
#pragma unroll
          for (int i = 0; i < Tl::WM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = fmaxf(mx, tile.acc[i][j][r]);
          if (s[j] != 0.0f) mx = fmaxf(mx, m[j]);
          mx = mx == -__builtin_inff() ? 0.0f : mx;   // any finite reference leaves the sum 0
          if (!renew) mx = m[j];
          // (no sum yet: m is no maximum, and mx may lie far below it)
          if (s[j] != 0.0f) s[j] *= ex2((m[j] - mx) * c[j]);
          m[j] = mx;
          sum = sum_against(mx);
        }
        s[j] += sum;
      }
    }
#pragma unroll
    for (int j = 0; j < Tl::WN; ++j) m[j] = s[j] == 0.0f ? -__builtin_inff() : m[j];
    // the two halves of a lane pair hold other rows of the same token, and so
    // do the waves above one another
#pragma unroll
    for (int j = 0; j < Tl::WN; ++j) {
      const float mo = __shfl_xor(m[j], 32, 64), so = __shfl_xor(s[j], 32, 64);
      const float mx = fmaxf(m[j], mo), ref = mx == -__builtin_inff() ? 0.0f : mx;
      const float a = s[j] * ex2((m[j] - ref) * c[j]), b = so * ex2((mo - ref) * c[j]);
      if (half == 0) hand[wr][(wc * Tl::WN + j) * 32 + l32] = make_float2(mx, a + b);
    }
    __syncthreads();
    for (int e = tid; e < Tl::BN; e += Tl::NTHR) {
      float mx = hand[0][e].x;
#pragma unroll
      for (int w = 1; w < Tl::WR; ++w) mx = fmaxf(mx, hand[w][e].x);
      const float ref = mx == -__builtin_inff() ? 0.0f : mx;
      const float ce = factor(n0 + e);
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < Tl::WR; ++w) sum += hand[w][e].y * ex2((hand[w][e].x - ref) * ce);
      if (n0 + e < N) part[(n0 + e) * splits + split] = make_float2(mx, sum);
    }
    __syncthreads();
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// One wave per token: joins the splits' pairs; the target's logit is a plain
// fp32 dot product.  A target outside the vocabulary gives a NaN loss.
template <bool BF16>
__global__ void __launch_bounds__(256) k_loss_join(const float2* __restrict__ part, int splits, const void* __restrict__ x,
                                                   const void* __restrict__ W, const void* __restrict__ targets,
                                                   int target_bytes, int64_t N, int64_t V, int64_t d, float scale,
                                                   const LossUnits* __restrict__ units, const float* __restrict__ top_x,
                                                   int64_t ignore,
                                                   float* __restrict__ loss, float* __restrict__ lse) {
  using S = Storage<BF16 ? kBF16 : kF32>;
  const int64_t n = block_in_rows() * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (n >= N) return;
  const float back = BF16 ? 1.0f : units->iw * inverse_unit(top_x[n]), c = above_zero(scale * kLog2e * back);
  const int64_t t = target_of(targets, target_bytes, n);
  const bool in = t >= 0 && t < V;
  // the pairs are on their way while the dot product waits for the target
  constexpr int kHeld = 4;
  const float2* const mine = part + n * splits;
  float2 held[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    held[k] = lane + 64 * k < splits ? mine[lane + 64 * k] : make_float2(-__builtin_inff(), 0.0f);
  float dot = 0.0f;
  if (in && t != ignore) {
    const typename S::T* xr = static_cast<const typename S::T*>(x) + n * d;
    const typename S::T* wr = static_cast<const typename S::T*>(W) + t * d;
#pragma unroll 8
    for (int64_t i = lane; i < d; i += 64) dot = fmaf(S::load(xr + i), S::load(wr + i), dot);
    dot = wave_sum(dot);
  }
  float m = held[0].x;
#pragma unroll
  for (int k = 1; k < kHeld; ++k) m = fmaxf(m, held[k].x);
  for (int i = lane + 64 * kHeld; i < splits; i += 64) m = fmaxf(m, mine[i].x);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  const float ref = m == -__builtin_inff() ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) s += held[k].y * ex2((held[k].x - ref) * c);
  for (int i = lane + 64 * kHeld; i < splits; i += 64) s += mine[i].y * ex2((mine[i].x - ref) * c);
  s = wave_sum(s);
  if (lane == 0) {
    const float ln = logf(s);
    lse[n] = fmaf(ref * back, scale, ln);
    loss[n] = t == ignore ? 0.0f : in ? fmaf(fmaf(ref, back, -dot), scale, ln) : __builtin_nanf("");
  }
}

// ------------------------------------------------------------ backward ---

// dz (in units of its call) of the vocabulary tiles of a piece (first entry
// piece0, rows to be written up to piece1), stored by token rows ldz apart
// (fp32 data: every 32 high terms and their 32 low ones).  A lane holds four
// neighbouring entries of its token at a time and the other half of the wave
// the next four: a swap of the halves makes them eight, 16 bytes, a swap of the
// halves' halves puts 64 bytes of 16 tokens into four lanes of one register, and
// a permutation of the lanes puts these side by side (32768 x 512 x 8192: stores
// of 16 bytes a row in a quarter of a wave 354 us, this 336, and 345 since x has a
// copy of its own for dW, which leaves this one out of the caches; without any
// store 295, the products alone 245).
// bf16 data goes past the caches, so that W and x stay in them: 336 us and 283
// for the dx that reads it, against 340 and 299, though half lines count for
// more there (694 MB written for 537).  fp32 data, whose two terms fill a line,
// does not: 4096 x 256 x 32000 252, dx 215, dW 229 us against 287, 209, 225.
template <class Tl, bool BF16>
__global__ void __launch_bounds__(Tl::NTHR, 2) k_loss_dz(MmOperand W, MmOperand X, int64_t N, int64_t V, int64_t d,
                                                         const LossUnits* __restrict__ units, int64_t piece0,
                                                         int64_t piece1, int n_tok, const RowCoef* __restrict__ coef,
                                                         const RowFar* __restrict__ far,
                                                         const float* __restrict__ row_unit, uint16_t* __restrict__ dz,
                                                         int64_t ldz) {
  const bool odd = __builtin_amdgcn_readfirstlane(units->odd) != 0;
  // the loads are up to NST tiles ahead (tiles of one stage)
  constexpr int kRing = Tl::NST + 1;
  static_assert(sizeof(RowCoef) == 16 && Tl::BN % 64 == 0 && Tl::BN / 64 <= Tl::NW, "one coefficient load per wave");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Tl::LDS];
  __shared__ __attribute__((aligned(1024))) RowCoef coefs[kRing][Tl::BN];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / Tl::WC, wc = wave % Tl::WC;
  const uint32_t v_tiles = static_cast<uint32_t>((piece1 - piece0 + Tl::BM - 1) / Tl::BM);
  constexpr uint32_t kGroup = 8;   // vocabulary tiles that an XCD's workgroups share
  Tl tile;
  tile.open(lds, W, V, X, N, 0, d);
  Units lu(v_tiles * n_tok), cu(lu);
  int fill = 0;   // the tokens' coefficients come with the tile's first stage
  auto go_to = [&]() {
    uint32_t vt, tok;
    tile_of(lu.u, v_tiles, n_tok, kGroup, vt, tok);
    const int64_t n0 = static_cast<int64_t>(tok) * Tl::BN;
    tile.template seek<false, false>(piece0 + static_cast<int64_t>(vt) * Tl::BM, n0);
    int l = lane;
    asm volatile("" : "+v"(l));
    if (wave < Tl::BN / 64) mm_dma(coef + imin(n0 + wave * 64 + l, N - 1), mm_lds_addr(coefs[fill] + wave * 64));
    fill = fill + 1 == kRing ? 0 : fill + 1;
  };
  auto next = [&]() {
    lu.advance();
    if (lu.valid()) go_to();
  };
  if (!lu.valid()) return;
  go_to();
  tile.template prime<false, false>(next);
  constexpr int TERMS = BF16 ? 1 : 2;
  constexpr int kStores = std::min(63, Tl::WM * Tl::WN * 2 * TERMS);   // of a wave and whole tile
  bool whole = false;   // the tile before was
  for (int use = 0; cu.valid(); cu.advance(), use = use + 1 == kRing ? 0 : use + 1) {
    uint32_t vt, tok;
    tile_of(cu.u, v_tiles, n_tok, kGroup, vt, tok);
    const int64_t v0 = piece0 + static_cast<int64_t>(vt) * Tl::BM, n0 = static_cast<int64_t>(tok) * Tl::BN;
    tile.template multiply<false, false, false, true, kStores>(next, whole);
    uint8_t* const base = reinterpret_cast<uint8_t*>(dz + n0 * ldz + TERMS * (v0 - piece0));
    const int rows = static_cast<int>(imin(piece1 - v0, Tl::BM)), toks = static_cast<int>(imin(N - n0, Tl::BN));
    const int vocab_left = static_cast<int>(imin(V - v0, Tl::BM));
    whole = vocab_left == Tl::BM && toks == Tl::BN;
    // opaque, so that what follows from them is not kept in registers over the tiles
    int el = lane, first_row = wr * Tl::WM * 32;
    asm volatile("" : "+v"(el), "+s"(first_row));
    const int eh = el >> 5;
    // this lane's place in a store: token el / 4 of 16, entries 8 (el % 4) ..; they
    // are in the lane of that token and chunk (chunks 0, 16, 8, 24 by lane / 16)
    const int eb = 8 * (el & 3), et = el >> 2;
    const int from = 4 * (et + 16 * ((el & 3) == 1 ? 2 : (el & 3) == 2 ? 1 : el & 3));
    const uint32_t ld2 = static_cast<uint32_t>(2 * ldz);
    auto finish = [&](auto edge) {
      constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
      for (int j = 0; j < Tl::WN; ++j) {
        const int tl = (wc * Tl::WN + j) * 32 + (el & 31);
        const int tb = (wc * Tl::WN + j) * 32 + et;
        const uint32_t at_row = static_cast<uint32_t>(tb) * ld2 + 2 * eb;
        const RowCoef rc = coefs[use][tl];
        // the target's row of this tile (negative or past the tile: elsewhere)
        const int at = rc.target < 0 ? -1 : static_cast<int>(imax(imin(rc.target - v0, 1 << 20), -1));
        const float c = fabsf(rc.c);
        const bool negative = __builtin_amdgcn_ballot_w64(rc.c < 0.0f) != 0;
#pragma unroll
        for (int i2 = 0; i2 < Tl::WM; ++i2) {
          const int vb = first_row + i2 * 32;   // the block's first row of the tile
          float v[16];
#pragma unroll
          for (int r = 0; r < 16; ++r) v[r] = ex2(fmaf(tile.acc[i2][j][r], c, -rc.lse2));
          if (odd) {   // rows in units of their own; far tokens' exponents, at most 14 (twice the weight) whatever lse's rounding
            asm volatile("");
            const RowFar f = far[imin(n0 + tl, N - 1)];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 k = *reinterpret_cast<const float4*>(row_unit + v0 + vb + 8 * q + 4 * eh);
              const float of[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float a = tile.acc[i2][j][4 * q + r] * of[r];
                const float e = fmaf(fmaf(a, f.back, -f.lse), kLog2e, f.log2p);
                v[4 * q + r] = ex2(is_far(rc.lse2) ? fminf(e, kUnit + 1.0f) : fmaf(a, c, -rc.lse2));
              }
            }
          }
          if (negative) {
            asm volatile("");   // branches: rarely taken
#pragma unroll
            for (int r = 0; r < 16; ++r) v[r] = rc.c < 0.0f ? -v[r] : v[r];
          }
          if (__builtin_amdgcn_ballot_w64(at >= vb && at < vb + 32)) {
            asm volatile("");
            const int rel = at - vb - 4 * eh;
#pragma unroll
            for (int r = 0; r < 16; ++r) v[r] -= rel == 8 * (r >> 2) + (r & 3) ? rc.one : 0.0f;
          }
          if (EDGE && vb + 32 > vocab_left) {   // the columns past the vocabulary are zeros (dx sums over them)
            asm volatile("");
#pragma unroll
            for (int r = 0; r < 16; ++r)
              if (vb + 4 * eh + 8 * (r >> 2) + (r & 3) >= vocab_left) v[r] = 0.0f;
          }
#pragma unroll
          for (int t = 0; t < TERMS; ++t) {
            uint32_t w[4][2];
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float &x0 = v[4 * q + 2 * e], &x1 = v[4 * q + 2 * e + 1];
                const mm_f16x2 p{static_cast<_Float16>(x0), static_cast<_Float16>(x1)};
                w[q][e] = __builtin_bit_cast(uint32_t, p);
                if (!BF16 && t == 0) {   // what is left for the second term
                  x0 -= static_cast<float>(p[0]);
                  x1 -= static_cast<float>(p[1]);
                }
              }
            // entry 8 (lane / 32) + 16 (lane / 16 % 2) of the block, token 16 k + lane % 16
            mm_u32x4 o[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const auto a = __builtin_amdgcn_permlane32_swap(w[0][e], w[1][e], false, false);
              const auto b = __builtin_amdgcn_permlane32_swap(w[2][e], w[3][e], false, false);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const auto f = __builtin_amdgcn_permlane16_swap(a[h], b[h], false, false);
                o[0][2 * h + e] = f[0];
                o[1][2 * h + e] = f[1];
              }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[k][e] = __builtin_amdgcn_ds_bpermute(from, o[k][e]);
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (!EDGE || (tb + 16 * k < toks && vb + eb < rows)) {
                mm_u32x4* const to = reinterpret_cast<mm_u32x4*>(base + (at_row + 16 * k * ld2 + 2 * TERMS * vb + 64 * t));
                if constexpr (BF16) __builtin_nontemporal_store(o[k], to); else gstore(to, o[k]);
              }
          }
        }
      }
    };
    if (whole) finish(std::false_type{}); else finish(std::true_type{});
  }
}

// a sum of dx (or dW) from its units: dx's are the token's, of weight u, and the
// column's
template <bool IS_W>
__device__ __forceinline__ float loss_finish(float v, int shift, float u, float column, float scale) {
  if constexpr (IS_W)
    return ldexpf(v * scale, -shift - kUnit);
  else
    return v * column * (u * scale);
}
// a column's: wd is W 2^(14 - exponent), dz has 2^kUnit
__device__ __forceinline__ float column_back(uint32_t top) {
  return ldexpf(1.0f, exponent_of(__uint_as_float(top)) - 14 - kUnit);
}

// P[z][r][c] (+)= sum over k of slice z of A(r, k) B(c, k), fp32, C columns; or,
// with `out`, the last of the sums times its units, rounded once to out[r][c].
// One workgroup per tile and slice, neighbours on one XCD.
template <class Tl, bool TA, bool BF16>
__global__ void __launch_bounds__(Tl::NTHR, 2) k_loss_mm(MmOperand A, MmOperand B, int64_t R, int64_t C, int64_t K,
                                                         int64_t k_slice, int n_col, int slices, int add,
                                                         float* __restrict__ P, void* __restrict__ out,
                                                         const LossUnits* __restrict__ units,
                                                         const float* __restrict__ weight,
                                                         const uint32_t* __restrict__ columns,
                                                         const uint16_t* __restrict__ wide_b, float scale) {
  using T = typename Storage<BF16 ? kBF16 : kF32>::T;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Tl::LDS];
  const uint32_t u = Units(gridDim.x).u, tiles = gridDim.x / slices, z = u / tiles, ti = u - z * tiles;
  const int64_t c0 = static_cast<int64_t>(ti % n_col) * Tl::BN, r0 = static_cast<int64_t>(ti / n_col) * Tl::BM;
  const int64_t k0 = static_cast<int64_t>(z) * k_slice, k1 = imin(k0 + k_slice, K);
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, l32 = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / Tl::WC, wc = wave % Tl::WC;
  const int shift = units->shift;
  const float iw = units->iw;
  bool wide = false;
  if constexpr (!TA) {   // dx: W in units of its columns, where it has more than one
    wide = units->wide != 0;
    B.base = wide ? wide_b : B.base;
  }
  Tl tile;
  tile.open(lds, A, R, B, C, k0, k1);
  auto next = []() {};
  tile.template seek<TA, true>(r0, c0);
  tile.template prime<TA, true>(next);
  // a uniform base and 32-bit offsets within the tile
  uint8_t* const base = reinterpret_cast<uint8_t*>(P + (z * R + r0) * C + c0);
  const int rows = static_cast<int>(imin(R - r0, Tl::BM)), cols = static_cast<int>(imin(C - c0, Tl::BN));
  const uint32_t ldb = static_cast<uint32_t>(C) * 4;
  const int rl = wr * Tl::WM * 32 + 4 * half, cl = wc * Tl::WN * 32 + l32;
  const uint32_t at = rl * ldb + cl * 4;
  if (add) {   // the sums so far, loaded beside the first stage
#pragma unroll
    for (int i = 0; i < Tl::WM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int ri = 32 * i + 8 * (r >> 2) + (r & 3);
#pragma unroll
        for (int j = 0; j < Tl::WN; ++j)
          tile.acc[i][j][r] = rl + ri < rows && cl + 32 * j < cols
                                  ? *reinterpret_cast<const float*>(base + (at + ri * ldb + 128 * j))
                                  : 0.0f;
      }
  } else {
    tile.clear();
  }
  tile.template multiply<TA, true, true, true>(next);
  T* const obase = static_cast<T*>(out) + r0 * C + c0;
  const uint32_t oat = rl * static_cast<uint32_t>(C) + cl;
  auto stores = [&](auto kind) {   // 0: sums that go on, 1: finished ones, 2: as `out` says
    constexpr int KIND = decltype(kind)::value;
    float column[Tl::WN] = {};
    if constexpr (!TA && KIND == 1) {
#pragma unroll
      for (int j = 0; j < Tl::WN; ++j) column[j] = iw / (1 << kUnit);
      if (wide) {
#pragma unroll
        for (int j = 0; j < Tl::WN; ++j) column[j] = column_back(columns[imin(c0 + cl + 32 * j, C - 1)]);
      }
    }
#pragma unroll
    for (int i = 0; i < Tl::WM; ++i) {
      float u[16] = {};   // the rows' weights (there are some for a whole tile)
      if constexpr (!TA && KIND == 1) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 f = *reinterpret_cast<const float4*>(weight + r0 + rl + 32 * i + 8 * q);
          u[4 * q] = f.x, u[4 * q + 1] = f.y, u[4 * q + 2] = f.z, u[4 * q + 3] = f.w;
        }
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int ri = 32 * i + 8 * (r >> 2) + (r & 3);
#pragma unroll
        for (int j = 0; j < Tl::WN; ++j) {
          if (rl + ri < rows && cl + 32 * j < cols) {
            if (KIND == 1 || (KIND == 2 && out))
              obase[oat + ri * static_cast<uint32_t>(C) + 32 * j] =
                  Storage<BF16 ? kBF16 : kF32>::pack(loss_finish<TA>(tile.acc[i][j][r], shift, u[r], column[j], scale));
            else
              *reinterpret_cast<float*>(base + (at + ri * ldb + 128 * j)) = tile.acc[i][j][r];
          }
        }
      }
    }
  };
  // dx by a loop of its own for each (4096 x 256 x 32000 fp32: 213 us against 228 with one), dW by one for both
  // (5003 x 520 x 50021 bf16: 308 against 324)
  if constexpr (TA)
    stores(std::integral_constant<int, 2>{});
  else if (out)
    stores(std::integral_constant<int, 1>{});
  else
    stores(std::integral_constant<int, 0>{});
}

// out[i] = the sum over z, in order, of P[z][i], from its units, rounded once
template <bool BF16, bool IS_W>
__global__ void __launch_bounds__(256) k_loss_out(const float* __restrict__ P, int S, int64_t n, int64_t d,
                                                  const LossUnits* __restrict__ units,
                                                  const float* __restrict__ weight,
                                                  const uint32_t* __restrict__ columns, float scale,
                                                  typename Storage<BF16 ? kBF16 : kF32>::T* __restrict__ out) {
  const int64_t i = block_in_rows() * 256 + threadIdx.x;
  if (i >= n) return;
  float sum = 0.0f;
  for (int z = 0; z < S; ++z) sum += P[z * n + i];
  const int64_t r = IS_W ? 0 : i / d;
  const float column = IS_W ? 1.0f : units->wide ? column_back(columns[i - r * d]) : units->iw / (1 << kUnit);
  out[i] = Storage<BF16 ? kBF16 : kF32>::pack(
      loss_finish<IS_W>(sum, units->shift, IS_W ? 1.0f : weight[r], column, scale));
}

template <class T>
__global__ void __launch_bounds__(256) k_loss_zero(T* __restrict__ out, int64_t n) {
  const int64_t i = block_in_rows() * 256 + threadIdx.x;
  if (i < n) out[i] = T(0);
}

// ---------------------------------------------------------------- plan ---

constexpr int64_t kCus = 256;
constexpr size_t kPieceBytes = size_t(512) << 20;   // of dz

size_t up(size_t x) { return (x + 255) / 256 * 256; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Operands laid out anew: bf16 rows of no multiple of 8 (for the logits), and
// the fp16 terms (fp32 data: for every product; bf16: for dx and dW).
struct Plan {
  bool pad;
  int planes;            // terms of x, W and dz
  int64_t ldp;
  size_t units_off, topx_off, topw_off, row_off, col_off, weight_off, xp_off, wp_off, xh_off, xg_off, wh_off, wd_off, end;
};
// Rows laid out anew are whole lines of 128 bytes, or an even part of one: a
// stage reads 128 bytes of every row, which other rows have in two lines (a
// forward call of 5003 x 1001 x 50021 took 587 us with rows of 2016 bytes and
// takes 534).  bf16 rows of a multiple of 8 are read where they are: at
// 5003 x 520 x 50021 the copy costs what it gains, 323 us to 318.
int64_t row_of(int64_t d, bool pair) {
  if (pair) return cdiv(d, 32) * 32;   // of both terms
  for (int64_t n = 8; n < 64; n *= 2)
    if (d <= n) return n;
  return cdiv(d, 64) * 64;
}
Plan plan_operands(const LossArgs& a, bool back) {
  Plan p{};
  p.planes = a.bf16 ? 1 : 2;
  const bool terms = back || !a.bf16;
  p.pad = !terms && a.d % 8 != 0;
  p.ldp = row_of(a.d, !a.bf16);
  size_t off = 0;
  auto take = [&](bool on, size_t bytes) {
    const size_t at = off;
    if (on) off += up(bytes);
    return at;
  };
  p.units_off = take(terms, sizeof(LossUnits));
  p.topx_off = take(terms, size_t(a.N) * 4);
  p.topw_off = take(terms, size_t(a.V) * 4);
  p.row_off = take(terms, size_t(cdiv(a.V, kBM)) * kBM * 4);   // whole tiles
  p.col_off = take(back, size_t(p.ldp) * 4);
  p.weight_off = take(back, size_t(cdiv(a.N, kBM)) * kBM * 4);
  p.xp_off = take(p.pad, size_t(a.N) * p.ldp * 2);
  p.wp_off = take(p.pad, size_t(a.V) * p.ldp * 2);
  p.xh_off = take(terms, size_t(p.planes) * a.N * p.ldp * 2);
  p.xg_off = take(back, size_t(p.planes) * a.N * p.ldp * 2);
  p.wh_off = take(terms, size_t(p.planes) * a.V * p.ldp * 2);
  p.wd_off = take(back, size_t(p.planes) * a.V * p.ldp * 2);
  p.end = off;
  return p;
}

// The logits' tile: Mid takes about 1.15 times Big's time per product (16384 x
// 512 x 16384: 285 and 245 us), which pays where 256 tokens a tile would waste
// more (100 x 512 x 32768: 16 and 21 us, fp32 60 and 73).
bool take_big(int64_t cols) { return cdiv(cols, kBig) * kBig * 100 <= cdiv(cols, kMid) * kMid * 115; }

struct PlanFw {
  Plan op;
  int kind;   // 0 Few, 1 Mid, 2 Big
  int64_t n_tok, splits, per_split, grid;
  size_t part_off, total;
};
PlanFw plan_fw(const LossArgs& a) {
  PlanFw f{};
  f.op = plan_operands(a, false);
  f.kind = a.N <= kFewN ? 0 : take_big(a.N) ? 2 : 1;
  const int64_t bm = f.kind == 0 ? kFewM : kBM, bn = f.kind == 0 ? kFewN : f.kind == 1 ? kMid : kBig;
  f.n_tok = cdiv(a.N, bn);
  const int64_t v_tiles = cdiv(a.V, bm), slots = (f.kind == 2 ? 1 : f.kind == 1 ? mid_slots(a.bf16) : 2) * kCus;
  // the number of splits whose longest workgroup has the fewest tiles, among
  // a few and the ones that fill whole rounds of the device
  int64_t best = -1;
  for (int64_t r = 1; r <= 8; ++r) {
    const int64_t want = r <= 4 ? r : (r - 4) * slots / f.n_tok;
    if (want < 1) continue;
    const int64_t per = cdiv(v_tiles, std::min(v_tiles, want)), s = cdiv(v_tiles, per);
    const int64_t longest = cdiv(f.n_tok * s, slots) * per;
    if (best < 0 || longest < best) {
      best = longest;
      f.splits = s;
      f.per_split = per;
    }
  }
  f.grid = std::min(f.n_tok * f.splits, slots);
  f.part_off = f.op.end;
  f.total = f.part_off + up(size_t(f.splits) * a.N * sizeof(float2));
  return f;
}

// A product's work: the rows whose tiles fill whole rounds of the device run
// over the whole sum each; the sum of the rest is cut in slices, joined after.
// The fewest microseconds of a few slice counts, with and without a head.
struct Cut {
  int64_t head;       // rows of the first kind
  int64_t s, len;     // slices of the rest's sum, and their length
};
Cut cut_of(int64_t rows, int64_t K, int64_t d, int terms, int64_t bn, double* us) {
  // microseconds of a CU for a tile over k of the sum (256 x 256 at 1.05
  // PFLOP/s of the device), and of storing fp32 sums and reading them again at
  // 4 TB/s, weighed half as much again: CUs that idle in a round leave the others
  // their power (16384 x 520 x 16384 with dx's 192 tiles in four slices of the
  // sum took 1093 us, in one 1066; 5003 x 520 x 50021 without the rest's slices
  // 1056, with them 1016)
  auto tile = [&](int64_t k) { return double(k) * terms * kBM * bn * (bn == kBig ? 1.0 : 1.12) * 2 / 4.1e6; };
  auto join = [&](int64_t n, int64_t s) { return s > 1 ? 4 + double(s) * n * d * 8 * 1.5 / 4e6 : 0.0; };
  const int64_t n_col = cdiv(d, bn), blocks = cdiv(rows, kBM), whole = blocks * n_col / kCus * kCus;
  Cut best{};
  *us = -1;
  for (int64_t head = 0;; head = std::min(whole / n_col * kBM, rows)) {
    const int64_t rest = rows - head, tiles = cdiv(rest, kBM) * n_col;
    const double first = cdiv(cdiv(head, kBM) * n_col, kCus) * tile(K) + (head > 0 && rest > 0 ? 3 : 0);
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

struct PlanBw {
  Plan op;
  bool big_z;               // tile of the logits
  int64_t out;              // tile columns of dx and dW
  int64_t piece, ldz;
  Cut x, w;                 // of dx's sum (over the piece), and dW's (over the tokens)
  size_t coef_off, far_off, dz_off, px_off, pw_off, total;
};
PlanBw plan_bw(const LossArgs& a) {
  PlanBw b{};
  b.op = plan_operands(a, true);
  b.big_z = take_big(a.N);
  const int64_t v_tiles = cdiv(a.V, kBM);
  const size_t row = size_t(a.N) * b.op.planes * 2 * kBM;
  int64_t per = std::max<int64_t>(1, int64_t(kPieceBytes / row));
  per = cdiv(v_tiles, cdiv(v_tiles, per));
  b.piece = per * kBM;
  // rows of dz are no power of two apart: they would fall on few memory channels
  b.ldz = b.op.planes * b.piece + 64;
  // the products' tile: the shorter of the two plans.  256 columns a tile are
  // faster than 192 per column, those waste less at the edge and may fill the
  // device's rounds better: 16384 x 520 x 16384 takes 1127 us with 192 and 1251
  // with 256, x 512 1025 and 873.  (128, two workgroups a CU, was never faster
  // than 192: dz is read once for every column of tiles.)
  const int64_t nv = std::min(b.piece, a.V);
  const int terms = a.bf16 ? 1 : kTerms;
  double best = -1;
  for (int64_t bn : {kBig, kWide}) {
    double tx, tw;
    const Cut x = cut_of(a.N, nv, a.d, terms, bn, &tx), w = cut_of(nv, a.N, a.d, terms, bn, &tw);
    if (best >= 0 && tx + tw >= best) continue;
    best = tx + tw;
    b.out = bn, b.x = x, b.w = w;
  }
  auto sums = [&](int64_t rows, const Cut& c) { return up((size_t(c.head) + size_t(c.s) * (rows - c.head)) * a.d * 4); };
  b.coef_off = b.op.end;
  b.far_off = b.coef_off + up(size_t(a.N) * sizeof(RowCoef));
  b.dz_off = b.far_off + up(size_t(a.N) * sizeof(RowFar));
  b.px_off = b.dz_off + up(size_t(a.N) * b.ldz * 2);
  b.pw_off = b.px_off + sums(a.N, b.x);
  b.total = b.pw_off + (b.w.s > 1 ? sums(nv, b.w) : 0);
  return b;
}

// The operands: X and Wo of the logits, Wo or (a W of more than one unit) Wd of dx
// (with dx_too) and Xg of dW (fp16 terms); with `coef`, the tokens' coefficients.  For the forward dloss ..
// far are null.
struct Operands {
  MmOperand X, Wo, Xg, Wd;
  LossUnits* units;
  float *top_x, *top_w, *row, *weight;
  uint32_t* col;
};
Operands lay_out(const LossArgs& a, const Plan& p, const void* x, const void* W, const void* targets, const float* lse,
                 const float* dloss, const float* dlse, RowCoef* coef, RowFar* far, bool dx_too) {
  Operands o{};
  auto at = [&](size_t off) { return reinterpret_cast<uint16_t*>(a.ws + off); };
  if (coef || !a.bf16) {
    auto parts = [](int64_t n) { return int(std::min<int64_t>(kMaxParts, cdiv(n, 256))); };
    o.units = reinterpret_cast<LossUnits*>(a.ws + p.units_off);
    o.top_x = reinterpret_cast<float*>(a.ws + p.topx_off);
    o.top_w = reinterpret_cast<float*>(a.ws + p.topw_off);
    o.weight = reinterpret_cast<float*>(a.ws + p.weight_off);
    o.X = {at(p.xh_off), p.planes * p.ldp};
    o.Xg = {at(p.xg_off), p.planes * p.ldp};
    o.Wo = {at(p.wh_off), p.planes * p.ldp};
    o.Wd = {at(p.wd_off), p.planes * p.ldp};
    o.row = reinterpret_cast<float*>(a.ws + p.row_off);
    o.col = dx_too ? reinterpret_cast<uint32_t*>(a.ws + p.col_off) : nullptr;
    const int lanes = a.d <= 128 ? 16 : a.d <= 256 ? 32 : 64;
    const int p1 = parts(a.N * lanes), p2 = parts(cdiv(a.V * a.d, 8));
    const int64_t n1 = cdiv(a.N * (p.ldp / 8), 256), n2 = cdiv(a.V * (p.ldp / 8), 256);
    auto go = [&](auto bf) {
      constexpr bool BF = decltype(bf)::value;
      k_loss_maxima<BF><<<unsigned(p1 + p2), 256, 0, a.stream>>>(dloss, dlse, targets, a.target_bytes, a.ignore, a.N, a.V,
                                                                 a.d, p.ldp, x, W, p1, lanes, p2, o.units, o.top_x, o.col);
      const int64_t blocks = cdiv(a.d, 256), share = cdiv(cdiv(a.V, std::max<int64_t>(1, 128 / blocks)), 32) * 32;
      const int64_t rows = std::min<int64_t>(128, cdiv(a.V * lanes, 1024)), cols = dx_too ? blocks * cdiv(a.V, share) : 0;
      k_loss_units<BF><<<unsigned(rows + cols), 1024, 0, a.stream>>>(W, a.V, a.d, int(rows), lanes, int(blocks), share, o.units,
                                                                     p1, p2, coef != nullptr, o.top_w, o.col);
      k_loss_layout<BF><<<rows_of_blocks(n1 + n2), 256, 0, a.stream>>>(
          dloss, dlse, lse, targets, a.target_bytes, a.ignore, a.N, a.V, a.d, a.scale, p.ldp, x, W, int(n1),
          o.units, o.top_x, o.top_w, o.row, o.col, o.weight, coef, far, at(p.xh_off), coef ? at(p.xg_off) : nullptr, at(p.wh_off),
          dx_too ? at(p.wd_off) : nullptr);
    };
    if (a.bf16) go(std::true_type{}); else go(std::false_type{});
  }
  if (o.units) return o;
  if (p.pad) {
    auto pad = [&](const void* in, int64_t R, size_t off) {
      k_loss_pad<<<rows_of_blocks(cdiv(R * (p.ldp / 8), 256)), 256, 0, a.stream>>>(static_cast<const uint16_t*>(in), R, a.d, p.ldp,
                                                                             at(off));
      return MmOperand{at(off), p.ldp};
    };
    o.X = pad(x, a.N, p.xp_off);
    o.Wo = pad(W, a.V, p.wp_off);
  } else {
    o.X = {static_cast<const uint16_t*>(x), a.d};
    o.Wo = {static_cast<const uint16_t*>(W), a.d};
  }
  return o;
}

}  // namespace

bool loss_fits(const LossArgs& a) {
  // rows x 16-byte chunks of the operands, and tiles of the logits
  const double tiles = double(cdiv(a.N, kFewN)) * double(cdiv(a.V, kFewM));
  const double lay = double(std::max(a.N, a.V)) * double(a.d / 8 + 1) / 256, out = double(std::max(a.N, a.V)) * double(a.d) / 256;
  return std::max({tiles, lay, out}) < 2147483647.0;
}
size_t loss_workspace(const LossArgs& a) { return a.N ? plan_fw(a).total : 0; }
size_t loss_backward_workspace(const LossArgs& a) { return a.N ? plan_bw(a).total : 0; }

void launch_loss(const LossArgs& a, const void* x, const void* W, const void* targets, float* loss, float* lse) {
  const PlanFw f = plan_fw(a);
  const Operands o = lay_out(a, f.op, x, W, targets, nullptr, nullptr, nullptr, nullptr, nullptr, false);
  const float c = a.scale * kLog2e;
  float2* part = reinterpret_cast<float2*>(a.ws + f.part_off);
  auto go = [&](auto pair) {
    constexpr bool PAIR = decltype(pair)::value;
    auto run = [&](auto tl) {
      using Tl = decltype(tl);
      k_loss_lse<Tl, PAIR><<<unsigned(f.grid), Tl::NTHR, 0, a.stream>>>(o.Wo, o.X, a.N, a.V, a.d, c, o.units, o.top_x, o.row, int(f.n_tok),
                                                                       int(f.splits), int(f.per_split), part);
    };
    if (f.kind == 0) run(Few<PAIR>{}); else if (f.kind == 1) run(Mid<PAIR>{}); else run(Big<PAIR>{});
  };
  if (a.bf16) go(std::false_type{}); else go(std::true_type{});
  const dim3 jg = rows_of_blocks(cdiv(a.N, 4));
  if (a.bf16)
    k_loss_join<true><<<jg, 256, 0, a.stream>>>(part, int(f.splits), x, W, targets, a.target_bytes, a.N, a.V, a.d,
                                                a.scale, o.units, o.top_x, a.ignore, loss, lse);
  else
    k_loss_join<false><<<jg, 256, 0, a.stream>>>(part, int(f.splits), x, W, targets, a.target_bytes, a.N, a.V, a.d,
                                                 a.scale, o.units, o.top_x, a.ignore, loss, lse);
}

void launch_loss_backward(const LossArgs& a, const void* x, const void* W, const void* targets, const float* lse,
                          const float* dloss, const float* dlse, void* dx, void* dW) {
  if (a.N == 0) {   // no token: dW is zero
    const int64_t n = a.V * a.d;
    if (dW && a.bf16)
      k_loss_zero<uint16_t><<<rows_of_blocks(cdiv(n, 256)), 256, 0, a.stream>>>(static_cast<uint16_t*>(dW), n);
    else if (dW)
      k_loss_zero<float><<<rows_of_blocks(cdiv(n, 256)), 256, 0, a.stream>>>(static_cast<float*>(dW), n);
    return;
  }
  const PlanBw b = plan_bw(a);
  RowCoef* coef = reinterpret_cast<RowCoef*>(a.ws + b.coef_off);
  RowFar* far = reinterpret_cast<RowFar*>(a.ws + b.far_off);
  uint16_t* dz = reinterpret_cast<uint16_t*>(a.ws + b.dz_off);
  float* px = reinterpret_cast<float*>(a.ws + b.px_off);
  float* pw = reinterpret_cast<float*>(a.ws + b.pw_off);
  const Operands o = lay_out(a, b.op, x, W, targets, lse, dloss, dlse, coef, far, dx != nullptr);
  LossUnits* const units = o.units;
  auto out = [&](auto bf, auto is_w, const float* P, int S, int64_t n, const float* weight, void* to) {
    constexpr bool BF = decltype(bf)::value, IS_W = decltype(is_w)::value;
    k_loss_out<BF, IS_W><<<rows_of_blocks(cdiv(n, 256)), 256, 0, a.stream>>>(P, S, n, a.d, units, weight, o.col, a.scale,
                                                                       static_cast<typename Storage<BF ? kBF16 : kF32>::T*>(to));
  };
  auto typed = [&](auto run) {
    if (a.bf16) run(std::true_type{}); else run(std::false_type{});
  };
  const size_t elt = a.bf16 ? 2 : 4;
  for (int64_t v0 = 0; v0 < a.V; v0 += b.piece) {
    const int64_t v1 = std::min(v0 + b.piece, a.V), nv = v1 - v0;
    const bool last = v1 == a.V;
    // dz rows reach the end of the piece's last tile of 8: zeros past the vocabulary
    const int64_t pend = v0 + cdiv(nv, 8) * 8;
    typed([&](auto bf) {
      constexpr bool BF = decltype(bf)::value;
      auto run = [&](auto tl) {
        using Tl = decltype(tl);
        const int64_t n_tok = cdiv(a.N, Tl::BN), tiles = n_tok * cdiv(nv, kBM), slots = (b.big_z ? 1 : mid_slots(BF)) * kCus;
        k_loss_dz<Tl, BF><<<unsigned(std::min(tiles, slots)), Tl::NTHR, 0, a.stream>>>(
            o.Wo, o.X, a.N, a.V, a.d, units, v0, pend, int(n_tok), coef, far, o.row, dz, b.ldz);
      };
      if (b.big_z) run(Big<!BF>{}); else run(Mid<!BF>{});
    });
    const MmOperand Z{dz, b.ldz};
    // head rows, then the rest, of a product whose rows lie `step` apart in Z
    auto product = [&](auto ta, const Cut& c, int64_t step, const MmOperand& B, const uint16_t* wide_b, int64_t rows,
                       int64_t K, bool add, float* P, bool finish, void* to) {
      constexpr bool TA = decltype(ta)::value;
      auto part = [&](int64_t r0, int64_t n, int64_t s, int64_t len, float* sums) {
        if (n <= 0) return;
        MmOperand A = Z;
        A.base += r0 * step;
        uint8_t* const dst = static_cast<uint8_t*>(to) + size_t(r0) * a.d * elt;
        typed([&](auto bf) {
          constexpr bool BF = decltype(bf)::value;
          auto run = [&](auto tl) {
            using Tl = decltype(tl);
            const int64_t n_col = cdiv(a.d, Tl::BN);
            k_loss_mm<Tl, TA, BF><<<unsigned(cdiv(n, kBM) * n_col * s), Tl::NTHR, 0, a.stream>>>(
                A, B, n, a.d, K, len, int(n_col), int(s), add, sums, finish && s == 1 ? dst : nullptr, units, o.weight + r0, o.col, wide_b, a.scale);
          };
          if (b.out == kBig) run(Big<!BF>{}); else run(Wide<!BF>{});
          if (finish && s > 1) out(bf, ta, sums, int(s), n * a.d, o.weight + r0, dst);
        });
      };
      const int64_t head = std::min(c.head, rows);
      part(0, head, 1, cdiv(K, 64) * 64, P);
      part(head, rows - head, c.s, c.len, P + head * a.d);
    };
    if (dx) {
      const MmOperand Wc{o.Wo.base + v0 * o.Wo.ld, o.Wo.ld};
      product(std::false_type{}, b.x, b.ldz, Wc, o.Wd.base + v0 * o.Wd.ld, a.N, nv, v0 > 0, px, last, dx);
    }
    if (dW) product(std::true_type{}, b.w, b.op.planes, o.Xg, nullptr, nv, a.N, false, pw, true, static_cast<uint8_t*>(dW) + v0 * a.d * elt);
  }
}

}  // namespace prn
