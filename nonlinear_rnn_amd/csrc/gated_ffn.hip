// Gated feed-forward product, and its gradients.
//
//   g = x Wg^T    u = x Wu^T    out = act(g) u        W = [Wg; Wu], 2 F x d
//   dg = dout u act'(g)         du = dout act(g)      dx = [dg | du] W      dW = [dg | du]^T x
//
// One kernel has both products: a tile of W is pairs of blocks of 32 rows, 32
// gate rows and the 32 up rows of the same outputs, so that the two sums of an
// output meet in one lane's accumulators, in fp32, and only the result is
// stored.  The backward pass forms the sums again (4 N F d operations) instead
// of reading 2 N F stored values, and stores dz = [dg | du], bf16: with its
// columns in the same pairs of blocks, 64 consecutive columns are 32 of dg and
// their 32 of du; dx and dW are one launch.
//
// Products run on the tiles of mm_tile.h, 256 x 256 in persistent workgroups
// where there are enough of them, else 128 x 128, two workgroups a CU.
//
// bf16: with the quarter tiles dz has two bf16 terms, v = hi + lo to 2^-16 |v|,
// and dx and dW are as exact as their own rounding lets them be (0.00166 of
// their root mean square against float64); the large ones round it once, and
// the errors of its entries, which meet at random, make that 0.00235: the
// second term would cost them a good part of a product's time (gradients of
// 5003 x 517 x 1387: 86 us, with two terms 119; of 32768 x 512 x 2048: 440 and 759).
//
// fp32: x, W and dz as three bf16 terms each, laid out before the products, six
// products of terms (bf16split.h), one pass of a tile over the sum each.  The
// forward runs on the projection's tiles, which split what they have in
// registers: one product alone does not pay for the layout (4096 x 256 x 704: 27
// us, in terms 38), three and their operands of either orientation do (the
// gradients 93 us; on the projection's tiles, with transposed copies, 118).
#include "gated_ffn.h"

#include <algorithm>
#include <type_traits>

#include "bf16split.h"
#include "gated_cell.h"
#include "gated_few.h"
#include "grid_rows.h"
#include "mm_plan.h"
#include "mm_tile.h"
#include "prn_device.h"
#include "proj.h"

namespace prn {
namespace {

// 8 waves, 256 x 256, 128 KB; 8 waves, 256 x 192, 112 KB; 4 waves, 128 x 128, 64 KB, two workgroups a CU (mm_tile.h)
using Big = MmTile<2, 4, 4, 2, 64, 2>;
using Wide = MmTile<4, 2, 2, 3, 64, 2>;
using Mid = MmTile<2, 2, 2, 2, 64, 2>;

// Copies of rows of d values as rows of ldp, zeros past d, a thread per 16 bytes:
// x (N rows) to xp, then W (two halves of F rows) to wp, the halves Fw rows each,
// zeros past F.  Nx or Fw = 0: not that one.
template <class T>
__global__ void __launch_bounds__(256) k_ffn_pad(const T* __restrict__ x, int64_t Nx, const T* __restrict__ W, int64_t F,
                                                 int64_t Fw, int64_t d, int64_t ldp, T* __restrict__ xp, T* __restrict__ wp) {
  constexpr int V = 16 / sizeof(T);
  const int64_t C = ldp / V, i = block_in_rows() * 256 + threadIdx.x;
  int64_t to = i / C;
  const int64_t c0 = (i - to * C) * V;
  const bool is_x = to < Nx;
  if (!is_x) to -= Nx;
  if (!is_x && to >= 2 * Fw) return;
  const int64_t half = !is_x && to >= Fw, r = to - half * Fw;
  const bool there = is_x || r < F;
  const T* const from = is_x ? x + r * d + c0 : W + (half * F + r) * d + c0;
  T v[V];
  if (there && c0 + V <= d) {
    __builtin_memcpy(v, from, sizeof(v));   // aligned or not
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = there && c0 + e < d ? from[e] : T(0);
  }
  __builtin_memcpy(__builtin_assume_aligned((is_x ? xp : wp) + to * ldp + c0, 16), v, sizeof(v));
}

// fp32 rows as three bf16 terms (bf16split.h), planes Nx ldp of x apart, 2 Fw ldp of
// W; rows and zeros as above, a thread per eight values
__global__ void __launch_bounds__(256) k_ffn_terms(const float* __restrict__ x, int64_t Nx, const float* __restrict__ W, int64_t F,
                                                   int64_t Fw, int64_t d, int64_t ldp, uint16_t* __restrict__ xp,
                                                   uint16_t* __restrict__ wp) {
  const int64_t C = ldp / 8, i = block_in_rows() * 256 + threadIdx.x;
  int64_t to = i / C;
  const int64_t c0 = (i - to * C) * 8;
  const bool is_x = to < Nx;
  if (!is_x) to -= Nx;
  if (!is_x && to >= 2 * Fw) return;
  const int64_t half = !is_x && to >= Fw, r = to - half * Fw;
  const bool there = is_x || r < F;
  const float* const from = is_x ? x + r * d + c0 : W + (half * F + r) * d + c0;
  sp_f32x4 a, b;
  if (there && c0 + 8 <= d) {
    __builtin_memcpy(&a, from, 16);   // aligned or not
    __builtin_memcpy(&b, from + 4, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = there && c0 + e < d ? from[e] : 0.0f;
      b[e] = there && c0 + 4 + e < d ? from[4 + e] : 0.0f;
    }
  }
  sp_bf16x8 t[3];
  split3(a, b, t[0], t[1], t[2]);
#pragma unroll
  for (int k = 0; k < 3; ++k)
    *reinterpret_cast<sp_bf16x8*>((is_x ? xp + k * Nx * ldp : wp + k * 2 * Fw * ldp) + to * ldp + c0) = t[k];
}

// The passes of a product over its operands' terms (kSplitU, kSplitV), two bits each
__device__ __forceinline__ int term_of_a(int pass) { return 0x910 >> 2 * pass & 3; }
__device__ __forceinline__ int term_of_b(int pass) { return 0x184 >> 2 * pass & 3; }
static_assert(kSplitU[2] == 1 && kSplitU[4] == 1 && kSplitU[5] == 2 && kSplitU[0] + kSplitU[1] + kSplitU[3] == 0, "0x910");
static_assert(kSplitV[1] == 1 && kSplitV[3] == 2 && kSplitV[4] == 1 && kSplitV[0] + kSplitV[2] + kSplitV[5] == 0, "0x184");

// ---------------------------------------------------- blocks of values ----
// A block of 32 x 32 values of the accumulators (lane l: column l % 32, a token;
// value 4 q + e: row 8 q + 4 (l / 32) + e, an output) as bf16 in two registers
// of 16 bytes a lane, as memory has them: register k, lane l: token 16 k + l / 4,
// outputs 8 (l % 4) .. + 7, so that four lanes have 64 bytes of a token.  Swaps
// of the wave's halves and quarters put eight outputs of a token into one lane,
// a permutation of the lanes puts a token's four side by side; each is its own
// inverse but the last.
__device__ __forceinline__ int quarter(int c) { return c == 1 ? 2 : c == 2 ? 1 : c; }

struct Packed {
  mm_u32x4 o[2];
};
__device__ __forceinline__ Packed to_rows(const float (&v)[16]) {
  const int l = threadIdx.x & 63, from = 4 * ((l >> 2) + 16 * quarter(l & 3));
  uint32_t w[4][2];
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      typedef __attribute__((ext_vector_type(2))) __bf16 b2;
      w[q][e] = __builtin_bit_cast(uint32_t, b2{static_cast<__bf16>(v[4 * q + 2 * e]), static_cast<__bf16>(v[4 * q + 2 * e + 1])});
    }
  Packed p;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0][e], w[1][e], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[2][e], w[3][e], false, false);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const auto f = __builtin_amdgcn_permlane16_swap(a[h], b[h], false, false);
      p.o[0][2 * h + e] = f[0];
      p.o[1][2 * h + e] = f[1];
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) p.o[k][e] = __builtin_amdgcn_ds_bpermute(from, p.o[k][e]);
  return p;
}
__device__ __forceinline__ void from_rows(Packed p, float (&v)[16]) {
  const int l = threadIdx.x & 63, from = 4 * (4 * (l & 15) + quarter(l >> 4));
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) p.o[k][e] = __builtin_amdgcn_ds_bpermute(from, p.o[k][e]);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    uint32_t a[2], b[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const auto f = __builtin_amdgcn_permlane16_swap(p.o[0][2 * h + e], p.o[1][2 * h + e], false, false);
      a[h] = f[0];
      b[h] = f[1];
    }
    const auto lo = __builtin_amdgcn_permlane32_swap(a[0], a[1], false, false);
    const auto hi = __builtin_amdgcn_permlane32_swap(b[0], b[1], false, false);
    const uint32_t w[4] = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[4 * q + 2 * e] = __uint_as_float(w[q] << 16);
      v[4 * q + 2 * e + 1] = __uint_as_float(w[q] & 0xffff0000u);
    }
  }
}

// what v is above its bf16 value, 0 where that is not finite
__device__ __forceinline__ float second_term(float v) {
  const float rest = v - static_cast<float>(static_cast<__bf16>(v));
  return fabsf(rest) < __builtin_inff() ? rest : 0.0f;
}

// ---------------------------------------------------------------- sums ----

// The tiles of g and u, 128 outputs x 256 tokens each (quarter tiles: 64 x 128).
// TERMS = 0: out (N x F), bf16.  Else dz in TERMS bf16 terms, `low` elements apart
// (N x 2 Fp in pairs of blocks, rows ldo apart, zeros past F); with three the data
// is fp32, W and X in terms w_low and x_low apart.  W has Fw gate rows, then Fw up
// rows.  A group of 8 tiles of outputs by all tokens, walked down the outputs
// first, is a share of an XCD, whose L2 then holds the group's W.  (32768 x 512 x
// 2048: 152 us, dz 186; two workgroups a CU of 256 x 128, one's products under the
// other's epilogue: 158 and 197.)
template <class Tl, int TERMS>
__global__ void __launch_bounds__(Tl::NTHR, 2) k_ffn_sums(MmOperand W, int64_t w_low, MmOperand X, int64_t x_low, int64_t N,
                                                          int64_t F, int64_t Fw, int64_t K, bool silu,
                                                          const void* __restrict__ dout_, void* __restrict__ out_, int64_t ldo,
                                                          int64_t low) {
  constexpr bool BACK = TERMS > 0, FP32 = TERMS == 3;
  using T = std::conditional_t<FP32, float, uint16_t>;
  constexpr int kPasses = FP32 ? 6 : 1;
  const T* const dout = static_cast<const T*>(dout_);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Tl::LDS];
  static_assert(Tl::WM % 2 == 0, "pairs of blocks");
  constexpr int kPairs = Tl::BM / 2;   // outputs of a tile
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / Tl::WC, wc = wave % Tl::WC;
  const uint32_t f_tiles = static_cast<uint32_t>((F + kPairs - 1) / kPairs), n_tok = static_cast<uint32_t>((N + Tl::BN - 1) / Tl::BN);
  constexpr uint32_t kGroup = 8;
  Tl tile;
  tile.open(lds, W, 2 * Fw, X, N, 0, K);
  Units lu(f_tiles * n_tok), cu(lu);
  int pass = 0;
  auto go_to = [&]() {
    uint32_t ft, tok;
    tile_of(lu.u, f_tiles, n_tok, kGroup, ft, tok);
    const int64_t f0 = static_cast<int64_t>(ft) * kPairs, n0 = static_cast<int64_t>(tok) * Tl::BN;
    if constexpr (kPasses > 1) tile.B.base = X.base + term_of_b(pass) * x_low;
    tile.template seek<false, false>(0, n0);
    tile.ab = reinterpret_cast<const uint8_t*>(W.base + (kPasses > 1 ? term_of_a(pass) * w_low : 0) + f0 * W.ld);
    const int lim = static_cast<int>(imin(Fw - 1 - f0, kPairs));
#pragma unroll
    for (int p = 0; p < Tl::NLA; ++p) {   // rows in pairs of blocks; past the last output, the last one's
      int s, f;
      Tl::template source<false, Tl::BM>(wave * Tl::NLA + p, lane, s, f);
      const int row = min((s >> 6) * 32 + (s & 31), lim);
      tile.offa[p] = static_cast<uint32_t>((((s >> 5) & 1) * Fw + row) * W.ld + f) * 2;
    }
  };
  auto next = [&]() {
    if (kPasses == 1 || ++pass == kPasses) {
      pass = 0;
      lu.advance();
    }
    if (lu.valid()) go_to();
  };
  if (!lu.valid()) return;
  go_to();
  tile.template prime<false, false>(next);
  constexpr int kStores = Tl::WN * Tl::WM * (BACK ? 2 * TERMS : 1);   // of a wave and whole tile
  bool whole = false;   // the tile before was
  for (; cu.valid(); cu.advance()) {
    uint32_t ft, tok;
    tile_of(cu.u, f_tiles, n_tok, kGroup, ft, tok);
    const int64_t f0 = static_cast<int64_t>(ft) * kPairs, n0 = static_cast<int64_t>(tok) * Tl::BN;
    if constexpr (kPasses == 1) {
      tile.template multiply<false, false, false, false, kStores>(next, whole);
    } else {
      tile.clear();
      for (int t = 0; t < kPasses; ++t) tile.template multiply<false, false, true, false, kStores>(next, t == 0 && whole);
    }
    const int f_left = static_cast<int>(imin(F - f0, kPairs)), toks = static_cast<int>(imin(N - n0, Tl::BN));
    // opaque, so that what follows from it is not kept in registers over the tiles
    int el = lane;
    asm volatile("" : "+v"(el));
    const int fe = 8 * (el & 3), te = el >> 2;   // this lane's place in a block as memory has it
    auto finish = [&](auto edge) {
      constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
      for (int j = 0; j < Tl::WN; ++j) {
        const int t0 = (wc * Tl::WN + j) * 32 + te;
        // fp32 data as the accumulators have it
        const int tf = (wc * Tl::WN + j) * 32 + (el & 31), ff = 4 * (el >> 5);
        Packed dp[Tl::WM / 2];
        if constexpr (BACK && !FP32) {   // all of dout before the first use
#pragma unroll
          for (int i = 0; i < Tl::WM / 2; ++i) {
            const int fb = (wr * (Tl::WM / 2) + i) * 32 + fe;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int t = t0 + 16 * k;
              const T* const at = dout + (n0 + t) * F + f0 + fb;
              if (!EDGE || (t < toks && fb + 8 <= f_left)) {
                __builtin_memcpy(&dp[i].o[k], at, 16);   // aligned or not
              } else {
                uint16_t e8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) e8[e] = t < toks && fb + e < f_left ? at[e] : uint16_t(0);
                __builtin_memcpy(&dp[i].o[k], e8, 16);
              }
            }
          }
        }
#pragma unroll
        for (int i = 0; i < Tl::WM / 2; ++i) {
          const int fb = (wr * (Tl::WM / 2) + i) * 32;
          const mm_f32x16 g = tile.acc[2 * i][j], u = tile.acc[2 * i + 1][j];
          float a[16], b[16];
          if constexpr (BACK) {
            if constexpr (FP32) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int f = fb + 8 * q + ff;
                const T* const at = dout + (n0 + tf) * F + f0 + f;
                if (!EDGE || (tf < toks && f + 4 <= f_left)) {
                  __builtin_memcpy(&a[4 * q], at, 16);   // aligned or not
                } else {
#pragma unroll
                  for (int e = 0; e < 4; ++e) a[4 * q + e] = tf < toks && f + e < f_left ? at[e] : 0.0f;
                }
              }
            } else {
              from_rows(dp[i], a);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const float e = ex2(-kLog2e * g[r]), on = rcp(1.0f + e), off = e < __builtin_inff() ? e * on : 1.0f;
              const float d = a[r], value = silu ? g[r] * on : on;
              const float slope = silu ? on * fmaf(g[r], off, 1.0f) : on * off;
              a[r] = d * u[r] * slope;
              b[r] = d * value;
            }
            if (EDGE && fb + 32 > f_left) {   // dx sums over these columns
              const int rest = f_left - fb - 4 * (el >> 5);
#pragma unroll
              for (int r = 0; r < 16; ++r)
                if (8 * (r >> 2) + (r & 3) >= rest) a[r] = b[r] = 0.0f;
            }
          } else {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const float s = rcp(1.0f + ex2(-kLog2e * g[r]));
              a[r] = (silu ? g[r] * s : s) * u[r];
            }
          }
          if (EDGE && fb >= f_left) continue;
#pragma unroll
          for (int term = 0; BACK && term < TERMS; ++term) {
            if (term > 0) {
#pragma unroll
              for (int r = 0; r < 16; ++r) a[r] = second_term(a[r]), b[r] = second_term(b[r]);
            }
            const Packed pa = to_rows(a), pb = to_rows(b);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int t = t0 + 16 * k;
              if (EDGE && t >= toks) continue;
              uint16_t* const to = static_cast<uint16_t*>(out_) + term * low + (n0 + t) * ldo + 2 * (f0 + fb) + fe;
              gstore(reinterpret_cast<mm_u32x4*>(to), pa.o[k]);
              gstore(reinterpret_cast<mm_u32x4*>(to + 32), pb.o[k]);
            }
          }
          if constexpr (!BACK) {
            const Packed pa = to_rows(a);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int t = t0 + 16 * k;
              if (EDGE && t >= toks) continue;
              uint16_t* const to = static_cast<uint16_t*>(out_) + (n0 + t) * ldo + f0 + fb + fe;
              if (!EDGE || fb + fe + 8 <= f_left) {
                __builtin_memcpy(to, &pa.o[k], 16);   // aligned or not
              } else {
                uint16_t e8[8];
                __builtin_memcpy(e8, &pa.o[k], 16);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (fb + fe + e < f_left) to[e] = e8[e];
              }
            }
          }
        }
      }
    };
    whole = f_left == kPairs && toks == Tl::BN;
    if (whole) finish(std::false_type{}); else finish(std::true_type{});
  }
}

// ----------------------------------------------------------- dx and dW ----

// One of the two products, C columns: tiles x slices of its sum over K.  Block b
// of its own: a tile and a slice, neighbours on one XCD (blocks are dealt to the
// XCDs in turn).
struct FfnProduct {
  MmOperand A, B;
  int64_t b_low, R, K, len;
  uint32_t slices, blocks;
  float* P;        // the slices' sums, R x C each
  void* out;       // one slice: the result
  __device__ __forceinline__ uint32_t unit(uint32_t b) const {
    const uint32_t x = b % kXcd;
    return x * (blocks / kXcd) + min(x, blocks % kXcd) + b / kXcd;
  }
};

// P[z][r][c] = sum over k of slice z of A(r, k) B(c, k), fp32, or with one slice
// `out` the sums rounded once.  TA: dW, A(r, k) = dz(k, r), the rows r in pairs
// of blocks: of `out`, row (r / 32 % 2) F + r / 64 * 32 + r % 32, if below F in
// its half.  Otherwise dx, k in pairs of blocks: B's rows (W) are half a stage
// of 64 from the gate's, half from the up rows Fw further on.  dz has TERMS
// terms, `low` elements apart; with three (fp32) B has as many, b_low apart.
template <class Tl, bool TA, int TERMS>
__device__ __forceinline__ void ffn_product(uint8_t* lds, const FfnProduct& p, uint32_t u, int64_t C, int64_t F, int64_t Fw,
                                            int64_t low) {
  using S = Storage<TERMS == 3 ? kF32 : kBF16>;
  using T = typename S::T;
  const uint32_t n_col = static_cast<uint32_t>((C + Tl::BN - 1) / Tl::BN), tiles = p.blocks / p.slices, z = u / tiles, ti = u - z * tiles;
  const int64_t c0 = static_cast<int64_t>(ti % n_col) * Tl::BN, r0 = static_cast<int64_t>(ti / n_col) * Tl::BM;
  const int64_t k0 = static_cast<int64_t>(z) * p.len, k1 = imin(k0 + p.len, p.K), R = p.R;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, l32 = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / Tl::WC, wc = wave % Tl::WC;
  Tl tile;
  tile.open(lds, p.A, R, p.B, C, k0, k1);
  constexpr int kPasses = TERMS == 3 ? 6 : TERMS;
  int pass = 0;
  auto go_to = [&]() {
    tile.A.base = p.A.base + (TERMS == 3 ? term_of_a(pass) : pass) * low;
    tile.B = p.B;
    if constexpr (TERMS == 3) tile.B.base += term_of_b(pass) * p.b_low;
    tile.template seek<TA, true>(r0, c0);
    if constexpr (!TA) {
      static_assert(Tl::KS == 64, "a stage is a pair of blocks");
      tile.bb = reinterpret_cast<const uint8_t*>(tile.B.base + k0 / 2 * p.B.ld + c0);
#pragma unroll
      for (int q = 0; q < Tl::NLB; ++q) {
        int s, f;
        Tl::template source<true, Tl::BN>(wave * Tl::NLB + q, lane, s, f);
        if (s >= 32) tile.offb[q] += static_cast<uint32_t>((Fw - 32) * p.B.ld * 2);
      }
      tile.B.ld = p.B.ld / 2;   // a stage goes on by 32 rows of either half
    }
  };
  auto next = [&]() {
    if (++pass < kPasses) go_to();
  };
  go_to();
  tile.clear();
  tile.template prime<TA, true>(next);
  if constexpr (kPasses == 1)
    tile.template multiply<TA, true>(next);
  else
    for (int t = 0; t < kPasses; ++t) tile.template multiply<TA, true, true>(next);
  const int rows = static_cast<int>(imin(R - r0, Tl::BM)), cols = static_cast<int>(imin(C - c0, Tl::BN));
  const int rl = wr * Tl::WM * 32 + 4 * half, cl = wc * Tl::WN * 32 + l32;
#pragma unroll
  for (int i = 0; i < Tl::WM; ++i) {
    // the block's first row of `out`, and how many of its rows are there
    const int64_t rb = r0 + (wr * Tl::WM + i) * 32, f = rb / 64 * 32;
    const int64_t ob = TA ? ((rb >> 5) & 1) * F + f : rb;
    const int there = TA ? static_cast<int>(imin(F - f, 32)) : 32;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int ri = 8 * (r >> 2) + (r & 3);
#pragma unroll
      for (int j = 0; j < Tl::WN; ++j) {
        if (rl + 32 * i + ri >= rows || cl + 32 * j >= cols) continue;
        if (p.slices == 1) {
          if (4 * half + ri < there)
            static_cast<T*>(p.out)[(ob + 4 * half + ri) * C + c0 + cl + 32 * j] = S::pack(tile.acc[i][j][r]);
        } else {
          p.P[(z * R + r0 + rl + 32 * i + ri) * C + c0 + cl + 32 * j] = tile.acc[i][j][r];
        }
      }
    }
  }
}

// dx and dW in one launch, the longer units first (w_first: dW's)
template <class Tl, int TERMS>
__global__ void __launch_bounds__(Tl::NTHR, 2) k_ffn_grads(FfnProduct x, FfnProduct w, bool w_first, int64_t C, int64_t F,
                                                           int64_t Fw, int64_t low) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Tl::LDS];
  const uint32_t b = blockIdx.x, first = w_first ? w.blocks : x.blocks;
  if ((b < first) == w_first)
    ffn_product<Tl, true, TERMS>(lds, w, w.unit(w_first ? b : b - first), C, F, Fw, low);
  else
    ffn_product<Tl, false, TERMS>(lds, x, x.unit(w_first ? b - first : b), C, F, Fw, low);
}

// out = the sum over z, in order, of P[z], rounded once, of either product with
// more than one slice (nx, nw values, or 0), four values a thread; dW's rows as in
// ffn_product.  Blocks [0, bx) dx.
template <bool FP32>
__global__ void __launch_bounds__(256) k_ffn_join(FfnProduct x, int64_t nx, int64_t bx, FfnProduct w, int64_t nw, int64_t C,
                                                  int64_t F) {
  using St = Storage<FP32 ? kF32 : kBF16>;
  using T = typename St::T;
  const int64_t b = block_in_rows();
  const bool is_w = b >= bx;
  const int64_t n = is_w ? nw : nx, i = 4 * ((is_w ? b - bx : b) * 256 + threadIdx.x);
  if (i >= n) return;
  const float* const P = (is_w ? w.P : x.P) + i;
  T* const out = static_cast<T*>(is_w ? w.out : x.out);
  const int S = static_cast<int>(is_w ? w.slices : x.slices), left = static_cast<int>(imin(n - i, 4));
  float sum[4] = {};
  for (int z = 0; z < S; ++z) {
    float v[4];
    if (left == 4) {
      __builtin_memcpy(v, P + z * n, 16);   // aligned or not
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = e < left ? P[z * n + e] : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += v[e];
  }
  T o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = St::pack(sum[e]);
  if (!is_w) {
    if (left == 4) {
      __builtin_memcpy(__builtin_assume_aligned(out + i, sizeof(o)), o, sizeof(o));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) out[i + e] = o[e];
    }
    return;
  }
  int64_t r = i < (int64_t(1) << 32) ? static_cast<uint32_t>(i) / static_cast<uint32_t>(C) : i / C, c = i - r * C;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t f = r / 64 * 32 + r % 32;
    if (e < left && f < F) out[(((r >> 5) & 1) * F + f) * C + c] = o[e];
    if (++c == C) c = 0, ++r;
  }
}

template <class T>
__global__ void __launch_bounds__(256) k_ffn_zero(T* __restrict__ out, int64_t n) {
  const int64_t i = block_in_rows() * 256 + threadIdx.x;
  if (i < n) out[i] = T(0);
}

// ---------------------------------------------------------------- plan ----

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// Few rows are gated_few.hip's: as many of its workgroups of 64 rows and 16 outputs
// as one round of the device takes (bf16) or two (fp32, which takes the tiles
// longer).  us, few and the tiles: 64 x 512 x 1408 bf16 5.4 and 8.1, 128 tokens 7.4
// and 7.9, 192 10.6 and 8.2; fp32 64 tokens 7.6 and 29, 256 20 and 26, 512 27 and 27.
bool few_rows(const GatedFfnArgs& a) { return cdiv(a.N, 64) * cdiv(a.F, 16) <= (a.bf16 ? kCus : 2 * kCus); }

// The 256 x 256 tiles where at least 128 of them keep the device busy, or the
// quarter tiles.  us, quarter and large: 3000 x 512 x 1408 (132 tiles) out 17.5
// and 18.2, the gradients (with two terms of dz and one) 79 and 64; 8192 x 512 x
// 1408 31 and 33, 164 and 109; 5003 x 517 x 1387 36 and 33, 130 and 87.  fp32: from 192 on, and where a pass is long enough to hide the start
// of the next: 5003 x 517 x 1387 377 and 304, 16384 x 512 x 1024 663 and 582, but
// 8192 x 512 x 512 (128 tiles) 173 and 203, 16384 x 256 x 512 191 and 212.
bool big_tiles(const GatedFfnArgs& a) {
  const int64_t tiles = cdiv(a.N, Big::BN) * cdiv(a.F, Big::BM / 2);
  return a.bf16 ? tiles >= 128 : tiles >= 192 && a.d > 256;
}

// How dx and dW, whose units share a launch, are cut: tiles of BM x BN, and slices of their sums.
struct Slices {
  int64_t s, len;
};
struct Split {
  Slices x, w;
  bool w_first;
};
template <class Tl>
Split split_of(int64_t N, int64_t Z, int64_t d, int terms, double* us) {
  // Microseconds of a unit over k of the sum, as in cut_of (the device at 1.05
  // PFLOP/s, 256 x 192 tiles at less), and 2 to begin and end; of storing the
  // slices' sums and reading them again, at 4 TB/s and half as much again.
  constexpr int64_t kSlots = kCus * 8 / Tl::NW;
  auto unit = [&](int64_t k) { return 2 + double(k) * terms * Tl::BM * Tl::BN * (Tl::BN == Wide::BN ? 1.12 : 1.0) * 2 * (kSlots / kCus) / 4.1e6; };
  auto join = [&](int64_t rows, int64_t s) { return s > 1 ? double(s) * rows * d * 8 * 1.5 / 4e6 : 0.0; };
  const int64_t n_col = cdiv(d, Tl::BN), tx = cdiv(N, Tl::BM) * n_col, tw = cdiv(Z, Tl::BM) * n_col;
  constexpr int64_t kCounts[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32};
  auto cut = [](int64_t K, int64_t want) {
    const int64_t len = cdiv(cdiv(K, want), 64) * 64;
    return Slices{cdiv(K, len), len};
  };
  Split best{};
  *us = -1;
  for (int64_t a : kCounts) {
    if (a > 1 && Z / a < 128) break;
    const Slices x = cut(Z, a);
    for (int64_t b : kCounts) {
      if (b > 1 && N / b < 128) break;
      const Slices w = cut(N, b);
      const int64_t nx = tx * x.s, nw = tw * w.s;
      const double ux = unit(x.len), uw = unit(w.len), longer = std::max(ux, uw), all = (nx * ux + nw * uw) / kSlots;
      // whole rounds of equal units, or about half of one unit's time is lost at the end
      const double run = nx + nw <= kSlots ? longer : std::max(all + std::min(ux, uw) / 2, longer);
      const double t = run + (x.s > 1 || w.s > 1 ? 4 : 0) + join(N, x.s) + join(Z, w.s);
      if (*us >= 0 && t >= *us) continue;
      *us = t;
      best = {x, w, uw > ux};
    }
  }
  return best;
}

struct Plan {
  bool big;               // the large tiles
  bool pad_x, pad_w;      // x and W laid out anew: rows that are no multiple of 16 bytes; fp32: in terms; for dx W's halves of Fw rows
  int64_t ldp, Fw;
  size_t x_off, w_off;
  // backward
  int64_t Fp, ldz;        // dz: columns of either kind, elements from row to row
  int64_t low;            // elements from a term to the next
  bool wide;              // 256 x 192 for dx and dW
  Slices x, w;            // of their sums
  bool w_first;
  size_t z_off, px_off, pw_off, total;
};

Plan plan_of(const GatedFfnArgs& a, bool back) {
  Plan p{};
  // bytes of x and W laid out: fp32 for the backward, three terms
  const int64_t vec = a.bf16 || back ? 8 : 4, elt = a.bf16 ? 2 : back ? 6 : 4;
  p.big = big_tiles(a);
  p.ldp = cdiv(a.d, vec) * vec;
  p.Fp = cdiv(a.F, 32) * 32;
  p.pad_x = elt == 6 || a.d != p.ldp;
  p.pad_w = p.pad_x || (back && a.F != p.Fp);
  p.Fw = back ? p.Fp : a.F;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += up(bytes);
    return at;
  };
  if (p.pad_x) p.x_off = take(size_t(a.N) * p.ldp * elt);
  if (p.pad_w) p.w_off = take(size_t(2) * p.Fw * p.ldp * elt);
  if (back) {
    p.ldz = 2 * p.Fp + 64;   // rows are no power of two apart: they would fall on few memory channels
    const int64_t Z = 2 * p.Fp;
    const int terms = !a.bf16 ? 3 : p.big ? 1 : 2, passes = a.bf16 ? terms : 6;
    double us, us_wide = -1;
    Split cut = p.big ? split_of<Big>(a.N, Z, a.d, passes, &us) : split_of<Mid>(a.N, Z, a.d, passes, &us);
    if (p.big) {
      const Split wide = split_of<Wide>(a.N, Z, a.d, passes, &us_wide);
      p.wide = us_wide < us;
      if (p.wide) cut = wide;
    }
    p.x = cut.x, p.w = cut.w, p.w_first = cut.w_first;
    auto sums = [&](int64_t rows, const Slices& c) { return c.s > 1 ? size_t(c.s) * rows * a.d * 4 : 0; };
    p.low = a.N * p.ldz;
    p.z_off = take(size_t(terms) * p.low * 2);
    p.px_off = take(sums(a.N, p.x));
    p.pw_off = take(sums(Z, p.w));
  }
  p.total = off;
  return p;
}

struct Operands {
  MmOperand x, W;         // fp32: the first of three terms,
  int64_t x_low, w_low;   // this far apart
};
Operands lay_out(const GatedFfnArgs& a, const Plan& p, const void* x, const void* W) {
  uint16_t *const xp = reinterpret_cast<uint16_t*>(a.ws + p.x_off), *const wp = reinterpret_cast<uint16_t*>(a.ws + p.w_off);
  const int64_t Nx = p.pad_x ? a.N : 0, Fw = p.pad_w ? p.Fw : 0;
  const dim3 grid = rows_of_blocks(cdiv((Nx + 2 * Fw) * (p.ldp / 8), 256));
  if (!a.bf16)
    k_ffn_terms<<<grid, 256, 0, a.stream>>>(static_cast<const float*>(x), Nx, static_cast<const float*>(W), a.F, Fw, a.d, p.ldp, xp, wp);
  else if (Nx + Fw > 0)
    k_ffn_pad<<<grid, 256, 0, a.stream>>>(static_cast<const uint16_t*>(x), Nx, static_cast<const uint16_t*>(W), a.F, Fw, a.d,
                                          p.ldp, xp, wp);
  return {{p.pad_x ? xp : static_cast<const uint16_t*>(x), p.ldp}, {p.pad_w ? wp : static_cast<const uint16_t*>(W), p.ldp},
          a.N * p.ldp, 2 * p.Fw * p.ldp};
}

// fp32 out: the projection's tiles
void out_fp32(const GatedFfnArgs& a, const Plan& p, const float* x, const float* W, float* out) {
  float *const xp = reinterpret_cast<float*>(a.ws + p.x_off), *const wp = reinterpret_cast<float*>(a.ws + p.w_off);
  if (p.pad_x) {
    k_ffn_pad<<<rows_of_blocks(cdiv((a.N + 2 * a.F) * (p.ldp / 4), 256)), 256, 0, a.stream>>>(x, a.N, W, a.F, a.F, a.d, p.ldp, xp, wp);
    x = xp, W = wp;
  }
  launch_proj_gated(x, W, out, a.N, p.ldp, a.F, a.silu, a.stream);
}

void fill_zero(const GatedFfnArgs& a, void* out, int64_t n) {
  const dim3 grid = rows_of_blocks(cdiv(n, 256));
  if (a.bf16)
    k_ffn_zero<<<grid, 256, 0, a.stream>>>(static_cast<uint16_t*>(out), n);
  else
    k_ffn_zero<<<grid, 256, 0, a.stream>>>(static_cast<float*>(out), n);
}

// out (bf16), or with dout dz
void sums(const GatedFfnArgs& a, const Plan& p, const Operands& o, const void* dout, void* out, int64_t ldo) {
  auto go = [&](auto tl, auto terms) {
    using Tl = decltype(tl);
    const unsigned grid = unsigned(std::min(cdiv(a.N, Tl::BN) * cdiv(a.F, Tl::BM / 2), kCus * 8 / Tl::NW));
    k_ffn_sums<Tl, decltype(terms)::value><<<grid, Tl::NTHR, 0, a.stream>>>(o.W, o.w_low, o.x, o.x_low, a.N, a.F, p.Fw, p.ldp, a.silu,
                                                                            dout, out, ldo, p.low);
  };
  constexpr std::integral_constant<int, 0> none{};
  constexpr std::integral_constant<int, 1> one{};
  constexpr std::integral_constant<int, 2> two{};
  constexpr std::integral_constant<int, 3> three{};
  if (!dout) {
    if (p.big) go(Big{}, none); else go(Mid{}, none);
  } else if (a.bf16) {
    if (p.big) go(Big{}, one); else go(Mid{}, two);
  } else {
    if (p.big) go(Big{}, three); else go(Mid{}, three);
  }
}

}  // namespace

bool gated_ffn_fits(const GatedFfnArgs& a) {
  const double N = double(a.N) + 256, d = double(a.d), F = double(a.F), most = double(int64_t(1) << 37);
  // byte offsets into W of 32 bits; launches below 2^32 threads: 2^22 tiles of 256 x 128, also where they are of 128 x 128
  return 2 * (F + 256) * (d + 64) < 2147483648.0 && N * (F + 128) < most && N * (d + 128) < most;
}

bool gated_ffn_backward_fits(const GatedFfnArgs& a) {
  // byte offsets of 32 bits into the rows of dz, fewer than 4 (F + 64) bytes, that a tile of dx reads
  return std::min(a.N, kTileRows) * (a.F + 64) <= int64_t(1) << 30;
}

size_t gated_ffn_workspace(const GatedFfnArgs& a) { return a.N == 0 || few_rows(a) ? 0 : plan_of(a, false).total; }

void launch_gated_ffn(const GatedFfnArgs& a, const void* x, const void* W, void* out) {
  if (few_rows(a)) {
    launch_few_ffn(GatedFewArgs{a.bf16, a.N, a.F, a.d, x, W, a.stream}, a.silu, out);
    return;
  }
  const Plan p = plan_of(a, false);
  if (a.bf16)
    sums(a, p, lay_out(a, p, x, W), nullptr, out, a.F);
  else
    out_fp32(a, p, static_cast<const float*>(x), static_cast<const float*>(W), static_cast<float*>(out));
}

size_t gated_ffn_backward_workspace(const GatedFfnArgs& a) { return a.N ? plan_of(a, true).total : 0; }

void launch_gated_ffn_backward(const GatedFfnArgs& a, const void* x, const void* W, const void* dout, void* dx, void* dW) {
  if (a.N == 0) {   // no row: dW is zero
    if (dW) fill_zero(a, dW, 2 * a.F * a.d);
    return;
  }
  const Plan p = plan_of(a, true);
  const Operands o = lay_out(a, p, x, W);
  uint16_t* const dz = reinterpret_cast<uint16_t*>(a.ws + p.z_off);
  float *const px = reinterpret_cast<float*>(a.ws + p.px_off), *const pw = reinterpret_cast<float*>(a.ws + p.pw_off);
  sums(a, p, o, dout, dz, p.ldz);
  const MmOperand Z{dz, p.ldz};
  const int64_t Zp = 2 * p.Fp;
  FfnProduct to_x{Z, o.W, o.w_low, a.N, Zp, p.x.len, uint32_t(p.x.s), 0, px, dx};
  FfnProduct to_w{Z, o.x, o.x_low, Zp, a.N, p.w.len, uint32_t(p.w.s), 0, pw, dW};
  auto run = [&](auto tl, auto terms) {
    using Tl = decltype(tl);
    const int64_t n_col = cdiv(a.d, Tl::BN);
    if (dx) to_x.blocks = uint32_t(cdiv(a.N, Tl::BM) * n_col * p.x.s);
    if (dW) to_w.blocks = uint32_t(cdiv(Zp, Tl::BM) * n_col * p.w.s);
    k_ffn_grads<Tl, decltype(terms)::value><<<to_x.blocks + to_w.blocks, Tl::NTHR, 0, a.stream>>>(to_x, to_w, p.w_first, a.d, a.F,
                                                                                                  p.Fw, p.low);
  };
  constexpr std::integral_constant<int, 1> one{};
  constexpr std::integral_constant<int, 2> two{};
  constexpr std::integral_constant<int, 3> three{};
  if (a.bf16) {
    if (!p.big) run(Mid{}, two); else if (p.wide) run(Wide{}, one); else run(Big{}, one);
  } else {
    if (!p.big) run(Mid{}, three); else if (p.wide) run(Wide{}, three); else run(Big{}, three);
  }
  const int64_t nx = dx && p.x.s > 1 ? a.N * a.d : 0, nw = dW && p.w.s > 1 ? Zp * a.d : 0;
  if (nx + nw == 0) return;
  const int64_t bx = cdiv(nx, 1024);
  const dim3 grid = rows_of_blocks(bx + cdiv(nw, 1024));
  if (a.bf16)
    k_ffn_join<false><<<grid, 256, 0, a.stream>>>(to_x, nx, bx, to_w, nw, a.d, a.F);
  else
    k_ffn_join<true><<<grid, 256, 0, a.stream>>>(to_x, nx, bx, to_w, nw, a.d, a.F);
}

}  // namespace prn
