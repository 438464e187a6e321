// Products of few rows with a gated end: z_p = x W_p^T for the two or three
// parts of W, and act(z_0) z_1 or a step of the gated linear recurrence.
//
// What bounds them is the latency of reading W once.  A workgroup has 16 outputs
// of every part and up to 64 rows of x; its waves share the sum over k, every
// wave all of its loads under way before its first product: fragments of the
// 16 x 16 matrix instructions come straight from memory, 16 bytes a lane (lane
// l: row l % 16, the l / 16-th 16 bytes of a step's 64; x comes from the
// caches).  The waves' sums meet in LDS and are added in wave order.
//   bf16: v_mfma_f32_16x16x32_bf16, 32 k a step
//   fp32: v_mfma_f32_16x16x4_f32, exact fp32 products, 16 k a step: the e-th
//         instruction takes the e-th value of every lane, of W and x alike
// Result: lane l, value e: output 4 (l / 16) + e, row l % 16.
#include "gated_few.h"

#include <type_traits>

#include "gated_cell.h"
#include "prn_device.h"

namespace prn {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;

constexpr int kWaves = 8;
constexpr int kOuts = 16;   // outputs of a workgroup
constexpr int64_t kCus = 256;

// 16 bytes of a row from element k on, zeros past K
template <class T>
__device__ __forceinline__ f32x4 edge16(const T* row, int64_t k, int64_t K) {
  constexpr int V = 16 / sizeof(T);
  T v[V];
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = k + e < K ? row[k + e] : T(0);
  f32x4 q;
  __builtin_memcpy(&q, v, 16);
  return q;
}

template <int DT>
__device__ __forceinline__ f32x4 products(f32x4 w, f32x4 x, f32x4 acc) {
  if constexpr (DT == kBF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(w[e], x[e], acc, 0, 0, 0);
    return acc;
  }
}

// TB blocks of 16 rows of x.  STEP: of the recurrence (bias, state, out and out2), else act(z_0) z_1 (silu, out).
template <int DT, int PARTS, int TB, bool STEP>
__global__ void __launch_bounds__(64 * kWaves) k_few(const typename Storage<DT>::T* __restrict__ x,
                                                     const typename Storage<DT>::T* __restrict__ W, int64_t N, int64_t R,
                                                     int64_t K, bool silu, const float* __restrict__ bias,
                                                     const typename Storage<DT>::T* __restrict__ state,
                                                     typename Storage<DT>::T* __restrict__ out,
                                                     typename Storage<DT>::T* __restrict__ out2) {
  using ST = Storage<DT>;
  using T = typename ST::T;
  constexpr int V = 16 / sizeof(T), KS = 4 * V;   // values of a lane, and k, of a step
  __shared__ float red[kWaves][PARTS][TB][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kOuts, n0 = static_cast<int64_t>(blockIdx.y) * (16 * TB);
  const T *wp[PARTS], *xp[TB];
#pragma unroll
  for (int p = 0; p < PARTS; ++p) wp[p] = W + (p * R + imin(r0 + (lane & 15), R - 1)) * K;
#pragma unroll
  for (int b = 0; b < TB; ++b) xp[b] = x + imin(n0 + 16 * b + (lane & 15), N - 1) * K;
  f32x4 acc[PARTS][TB] = {};
  const int64_t kl = V * (lane >> 4), whole = K / KS;
  auto step = [&](const f32x4 (&w)[PARTS], const f32x4 (&v)[TB]) {
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
#pragma unroll
      for (int b = 0; b < TB; ++b) acc[p][b] = products<DT>(w[p], v[b], acc[p][b]);
  };
  auto load = [&](int64_t s, f32x4 (&w)[PARTS], f32x4 (&v)[TB]) {   // aligned or not
#pragma unroll
    for (int p = 0; p < PARTS; ++p) __builtin_memcpy(&w[p], wp[p] + s * KS + kl, 16);
#pragma unroll
    for (int b = 0; b < TB; ++b) __builtin_memcpy(&v[b], xp[b] + s * KS + kl, 16);
  };
  constexpr int U = 4;
  int64_t s = wave;
  for (; s + (U - 1) * kWaves < whole; s += U * kWaves) {
    f32x4 w[U][PARTS], v[U][TB];
#pragma unroll
    for (int u = 0; u < U; ++u) load(s + u * kWaves, w[u], v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) step(w[u], v[u]);
  }
  if (s + kWaves < whole) {
    f32x4 w[2][PARTS], v[2][TB];
    load(s, w[0], v[0]);
    load(s + kWaves, w[1], v[1]);
    step(w[0], v[0]);
    step(w[1], v[1]);
    s += 2 * kWaves;
  }
  for (; s * KS < K; s += kWaves) {
    f32x4 w[PARTS], v[TB];
    if (s < whole) {
      load(s, w, v);
    } else {
#pragma unroll
      for (int p = 0; p < PARTS; ++p) w[p] = edge16(wp[p], s * KS + kl, K);
#pragma unroll
      for (int b = 0; b < TB; ++b) v[b] = edge16(xp[b], s * KS + kl, K);
    }
    step(w, v);
  }
#pragma unroll
  for (int p = 0; p < PARTS; ++p)
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][p][b][e][lane] = acc[p][b][e];
  __syncthreads();
  // consecutive threads have consecutive outputs of a row
  for (int o = threadIdx.x; o < TB * 256; o += 64 * kWaves) {
    const int ro = o & 15, t = (o >> 4) & 15, b = o >> 8;
    const int64_t r = r0 + ro, n = n0 + 16 * b + t;
    if (r >= R || n >= N) continue;
    float z[PARTS];
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      float q[kWaves];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) q[w] = red[w][p][b][ro & 3][16 * (ro >> 2) + t];
      z[p] = q[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) z[p] += q[w];
      if constexpr (STEP) {
        if (bias) z[p] += bias[p * R + r];
      }
    }
    if constexpr (STEP) {
      const Gate f = gate_of(z[0]);
      const float in = PARTS == 2 ? f.off : gate_of(z[1]).on, h = state ? ST::load(state + n * R + r) : 0.0f;
      const T y = ST::pack(fmaf(f.on, h, in * z[PARTS - 1]));
      out[n * R + r] = y;
      if (out2) out2[n * R + r] = y;
    } else {
      const float on = gate_of(z[0]).on;
      out[n * R + r] = ST::pack((silu ? z[0] * on : on) * z[PARTS - 1]);
    }
  }
}

template <int PARTS, bool STEP>
void launch(const GatedFewArgs& a, bool silu, const float* bias, const void* state, void* out, void* out2) {
  auto go = [&](auto dt, auto tb) {
    constexpr int DT = decltype(dt)::value, TB = decltype(tb)::value;
    using T = typename Storage<DT>::T;
    const dim3 grid(unsigned((a.R + kOuts - 1) / kOuts), unsigned((a.N + 16 * TB - 1) / (16 * TB)));
    k_few<DT, PARTS, TB, STEP><<<grid, 64 * kWaves, 0, a.stream>>>(static_cast<const T*>(a.x), static_cast<const T*>(a.W), a.N, a.R, a.K,
                                                                   silu, bias, static_cast<const T*>(state), static_cast<T*>(out),
                                                                   static_cast<T*>(out2));
  };
  // The fewest rows of x a workgroup with which there is one for every CU at most:
  // more workgroups read x less often each, fewer read W less often in all (64 x 512
  // x 1408 bf16 in 16, 32, 64 rows: 5.0, 4.7, 6.6 us; 64 x 1024 x 4096: 12.9, 10.1, 9.3).
  auto blocks = [&](auto dt) {
    const int64_t outs = (a.R + kOuts - 1) / kOuts;
    auto fits = [&](int64_t tb) { return a.N <= 16 * tb || outs * ((a.N + 16 * tb - 1) / (16 * tb)) <= kCus; };
    if (fits(1))
      go(dt, std::integral_constant<int, 1>{});
    else if (fits(2))
      go(dt, std::integral_constant<int, 2>{});
    else
      go(dt, std::integral_constant<int, 4>{});
  };
  if (a.bf16) blocks(std::integral_constant<int, kBF16>{}); else blocks(std::integral_constant<int, kF32>{});
}

}  // namespace

void launch_few_ffn(const GatedFewArgs& a, bool silu, void* out) { launch<2, false>(a, silu, nullptr, nullptr, out, nullptr); }

void launch_few_step(const GatedFewArgs& a, int parts, const float* bias, const void* state_in, void* state_out, void* h_out) {
  if (parts == 2)
    launch<2, true>(a, false, bias, state_in, state_out, h_out);
  else
    launch<3, true>(a, false, bias, state_in, state_out, h_out);
}

}  // namespace prn
