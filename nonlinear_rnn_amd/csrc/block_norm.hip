// Norms before and after a block, with the block's gate and residual scale.
//
//   u = h rstd(h) w_post       rstd(y) = 1 / sqrt(mean(y^2) + eps)
//   v = u act(gate)            act: silu(g) = g sig(g), or sig(g)
//   r = x + alpha v
//   n = r rstd(r) w_pre
//
// Each of w_post, gate, x, alpha, w_pre may be absent (its step is then the
// identity).  One pass over the rows each way: a row lives in the registers
// of a group of TPR lanes, so the bound is the memory (forward: h, gate, x in,
// r, n out; backward: h, gate, x, dr, dn in, dh, dgate, dx out).  The backward
// pass recomputes the row (two short sums) rather than reading saved
// statistics and r.
//
// Backward, with rn = r rstd(r), hn = h rstd(h):
//   q = dn w_pre        R = dr + rstd(r) (q - rn mean(q rn))      (= dx)
//   dalpha = sum R v    dv = R alpha       dw_pre = sum dn rn
//   dgate = dv u act'(gate)                du = dv act(gate)
//   p = du w_post       dh = rstd(h) (p - hn mean(p hn))          dw_post = sum du hn
// sums over rows: every lane keeps its channels' sums over the rows of its
// group, the groups of a workgroup are added in order through LDS, the
// workgroups' partials in order by a second kernel (bitwise reproducible).
#include "block_norm.h"

#include <algorithm>

#include "prn_device.h"

namespace prn {
namespace {

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}
// sum over groups of 16 or 64 lanes, in every lane, without LDS: lanes l ^ 1,
// l ^ 2, the mirror images in 8 and 16 lanes, then the other rows and halves
template <int W>
__device__ __forceinline__ float lane_sum(float v) {
  v += dpp<0xb1>(v);
  v += dpp<0x4e>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  if constexpr (W == 64) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(b[0]) + __uint_as_float(b[1]);
  }
  return v;
}

// sums of M values over the TPR lanes of a row.  A row of several waves joins
// them through LDS; `slot` alternates, so that one barrier per sum is enough.
template <int TPR, int M>
struct RowSum {
  static constexpr int NW = TPR / 64;
  float (*red)[M][TPR > 64 ? TPR / 64 : 1];
  int slot = 0;
  __device__ __forceinline__ void operator()(float* v) {
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] = lane_sum<(TPR < 64 ? 16 : 64)>(v[i]);
    if constexpr (TPR > 64) {
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int i = 0; i < M; ++i) red[slot][i][threadIdx.x >> 6] = v[i];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < M; ++i) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) s += red[slot][i][w];
        v[i] = s;
      }
      slot ^= 1;
    }
  }
};

// VEC consecutive channels of a row
template <int DT, int VEC>
__device__ __forceinline__ void load_vec(const typename Storage<DT>::T* p, float* o) {
  if constexpr (VEC == 1) {
    o[0] = Storage<DT>::load(p);
  } else if constexpr (DT == kF32) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    o[0] = q.x, o[1] = q.y, o[2] = q.z, o[3] = q.w;
  } else {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[2 * e] = __uint_as_float(w[e] << 16);
      o[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
}
template <int DT, int VEC>
__device__ __forceinline__ void store_vec(typename Storage<DT>::T* p, const float* o) {
  if constexpr (VEC == 1) {
    *p = Storage<DT>::pack(o[0]);
  } else if constexpr (DT == kF32) {
    *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = Storage<kBF16>::pack(o[2 * e]) | static_cast<uint32_t>(Storage<kBF16>::pack(o[2 * e + 1])) << 16;
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

struct NormDev {
  const void *h, *gate, *x, *dr, *dn;
  void *o0, *o1, *o2;   // forward: r, n; backward: dh, dgate, dx
  const float *w_post, *w_pre, *alpha;
  float* part;          // backward: the workgroups' weight-gradient sums, 3 x G x d
  int64_t N;
  int d, act;
  float eps;
};

// A lane's channels: chunk v of VEC channels starts at (v TPR + lane) VEC.
template <int DT, int VEC, int NV, int TPR>
struct Row {
  static constexpr int E = VEC * NV;
  int lane, d;
  __device__ __forceinline__ int at(int v) const { return (v * TPR + lane) * VEC; }
  __device__ __forceinline__ void load(const void* p, int64_t row, float* o) const {
    const typename Storage<DT>::T* q = static_cast<const typename Storage<DT>::T*>(p) + row * d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (at(v) < d) {
        load_vec<DT, VEC>(q + at(v), o + v * VEC);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[v * VEC + e] = 0.0f;
      }
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t row, const float* o) const {
    typename Storage<DT>::T* q = static_cast<typename Storage<DT>::T*>(p) + row * d;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (at(v) < d) store_vec<DT, VEC>(q + at(v), o + v * VEC);
  }
  // fp32 weights of the lane's channels; absent: ones
  __device__ __forceinline__ void weights(const float* p, float* o) const {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < VEC; ++e) o[v * VEC + e] = (p && at(v) < d) ? p[at(v) + e] : 1.0f;
  }
};

__device__ __forceinline__ float sig(float g) { return rcp(1.0f + ex2(kSigScale * g)); }

template <int DT, int VEC, int NV, int TPR, int NTHR>
__global__ void __launch_bounds__(NTHR) k_block_norm(NormDev a) {
  using R = Row<DT, VEC, NV, TPR>;
  constexpr int E = R::E;
  __shared__ float red[2][1][TPR > 64 ? TPR / 64 : 1];
  const R row{static_cast<int>(threadIdx.x) % TPR, a.d};
  const int64_t n = static_cast<int64_t>(blockIdx.x) * (NTHR / TPR) + threadIdx.x / TPR;
  if (TPR <= 64 && n >= a.N) return;   // a row of several waves is the workgroup's only one
  RowSum<TPR, 1> total{red};
  const float inv_d = 1.0f / static_cast<float>(a.d);
  float h[E], g[E], x[E];
  row.load(a.h, n, h);
  if (a.gate) row.load(a.gate, n, g);
  if (a.x) row.load(a.x, n, x);
  if (a.w_post) {
    float s = 0.0f, w[E];
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(h[e], h[e], s);
    row.weights(a.w_post, w);
    total(&s);
    const float rstd = __builtin_amdgcn_rsqf(fmaf(s, inv_d, a.eps));
#pragma unroll
    for (int e = 0; e < E; ++e) h[e] *= rstd * w[e];
  }
  if (a.gate) {
#pragma unroll
    for (int e = 0; e < E; ++e) h[e] *= a.act == 0 ? g[e] * sig(g[e]) : sig(g[e]);
  }
  if (a.alpha) {
    float w[E];
    row.weights(a.alpha, w);
#pragma unroll
    for (int e = 0; e < E; ++e) h[e] *= w[e];
  }
  if (a.x) {
#pragma unroll
    for (int e = 0; e < E; ++e) h[e] += x[e];
  }
  if (a.o0) row.store(a.o0, n, h);
  if (a.w_pre) {
    float s = 0.0f, w[E];
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(h[e], h[e], s);
    row.weights(a.w_pre, w);
    total(&s);
    const float rstd = __builtin_amdgcn_rsqf(fmaf(s, inv_d, a.eps));
#pragma unroll
    for (int e = 0; e < E; ++e) h[e] *= rstd * w[e];
    row.store(a.o1, n, h);
  }
}

template <int DT, int VEC, int NV, int TPR, int NTHR>
__global__ void __launch_bounds__(NTHR) k_block_norm_backward(NormDev a) {
  using R = Row<DT, VEC, NV, TPR>;
  constexpr int E = R::E, GROUPS = NTHR / TPR;
  __shared__ float red1[2][1][TPR > 64 ? TPR / 64 : 1];
  __shared__ float red2[2][2][TPR > 64 ? TPR / 64 : 1];
  __shared__ float hand[GROUPS > 1 ? NTHR * E : 1];
  const R row{static_cast<int>(threadIdx.x) % TPR, a.d};
  RowSum<TPR, 1> total{red1};
  RowSum<TPR, 2> total2{red2};
  const float inv_d = 1.0f / static_cast<float>(a.d);
  float w_post[E], w_pre[E], alpha[E], s_post[E], s_pre[E], s_alpha[E];
  row.weights(a.w_post, w_post);
  row.weights(a.w_pre, w_pre);
  row.weights(a.alpha, alpha);
#pragma unroll
  for (int e = 0; e < E; ++e) s_post[e] = s_pre[e] = s_alpha[e] = 0.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * GROUPS;
  for (int64_t n = static_cast<int64_t>(blockIdx.x) * GROUPS + threadIdx.x / TPR; n < a.N; n += step) {
    float h[E], g[E], x[E], dr[E], dn[E];
    row.load(a.h, n, h);
    if (a.gate) row.load(a.gate, n, g);
    if (a.x) row.load(a.x, n, x);
    if (a.dr) {
      row.load(a.dr, n, dr);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) dr[e] = 0.0f;
    }
    if (a.w_pre) row.load(a.dn, n, dn);
    float rstd_h = 1.0f;
    if (a.w_post) {
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(h[e], h[e], s);
      total(&s);
      rstd_h = __builtin_amdgcn_rsqf(fmaf(s, inv_d, a.eps));
#pragma unroll
      for (int e = 0; e < E; ++e) h[e] *= rstd_h;
    }
    // h is hn from here on; u = hn w_post, f = act(gate)
    float f[E], v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      f[e] = 1.0f;
      if (a.gate) {
        const float sg = sig(g[e]);
        f[e] = a.act == 0 ? g[e] * sg : sg;
        // act'(g)
        g[e] = a.act == 0 ? sg * fmaf(g[e], 1.0f - sg, 1.0f) : sg * (1.0f - sg);
      }
      v[e] = h[e] * w_post[e] * f[e];
    }
    if (a.w_pre) {
      float s[2] = {0.0f, 0.0f}, r[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        r[e] = a.x ? fmaf(alpha[e], v[e], x[e]) : alpha[e] * v[e];
        s[0] = fmaf(r[e], r[e], s[0]);
        s[1] = fmaf(dn[e] * w_pre[e], r[e], s[1]);
      }
      total2(s);
      const float rstd = __builtin_amdgcn_rsqf(fmaf(s[0], inv_d, a.eps));
      const float mean = s[1] * rstd * inv_d;   // mean(q rn)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float rn = r[e] * rstd;
        s_pre[e] = fmaf(dn[e], rn, s_pre[e]);
        dr[e] = fmaf(rstd, fmaf(dn[e], w_pre[e], -rn * mean), dr[e]);
      }
    }
    if (a.o2) row.store(a.o2, n, dr);
    float dg[E];
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      s_alpha[e] = fmaf(dr[e], v[e], s_alpha[e]);
      const float dv = dr[e] * alpha[e];
      if (a.gate) dg[e] = dv * h[e] * w_post[e] * g[e];
      const float du = dv * f[e];
      s_post[e] = fmaf(du, h[e], s_post[e]);
      dr[e] = du * w_post[e];
      s = fmaf(dr[e], h[e], s);
    }
    if (a.o1) row.store(a.o1, n, dg);
    if (a.w_post) {
      total(&s);
      const float mean = s * inv_d;
#pragma unroll
      for (int e = 0; e < E; ++e) dr[e] = rstd_h * fmaf(-h[e], mean, dr[e]);
    }
    if (a.o0) row.store(a.o0, n, dr);
  }
  // the workgroup's sums: its groups in order
  for (int k = 0; k < 3; ++k) {
    if (!(k == 0 ? a.w_post : k == 1 ? a.w_pre : a.alpha)) continue;
    float* const out = a.part + (static_cast<int64_t>(k) * gridDim.x + blockIdx.x) * a.d;
    if constexpr (GROUPS > 1) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int i = v * VEC + e;
          hand[(threadIdx.x / TPR) * (TPR * E) + row.at(v) + e] = k == 0 ? s_post[i] : k == 1 ? s_pre[i] : s_alpha[i];
        }
      __syncthreads();
      for (int c = threadIdx.x; c < a.d; c += NTHR) {
        float s = 0.0f;
        for (int q = 0; q < GROUPS; ++q) s += hand[q * (TPR * E) + c];
        out[c] = s;
      }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int i = v * VEC + e;
          if (row.at(v) < a.d) out[row.at(v) + e] = k == 0 ? s_post[i] : k == 1 ? s_pre[i] : s_alpha[i];
        }
    }
  }
}

// out_k[c] = the sum over the G workgroups' partials: 16 waves take every
// 16th partial of 64 channels in order, their sums are added in order
__global__ void __launch_bounds__(1024) k_block_norm_weights(const float* __restrict__ part, int G, int d,
                                                             float* o0, float* o1, float* o2) {
  __shared__ float hand[16][64];
  const int k = blockIdx.y, lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
  float* const out = k == 0 ? o0 : k == 1 ? o1 : o2;
  if (!out) return;
  const float* p = part + static_cast<int64_t>(k) * G * d;
  float s = 0.0f;
  if (c < d) {
#pragma unroll 8
    for (int g = w; g < G; g += 16) s += p[static_cast<int64_t>(g) * d + c];
  }
  hand[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < d) {
#pragma unroll
    for (int q = 1; q < 16; ++q) s += hand[q][lane];
    out[c] = s;
  }
}

// lanes per row, chunks per lane, workgroup: at most 8 channels a lane (16
// take the backward pass past 256 registers)
struct Geo {
  int tpr, nv, nthr;
  bool vec;
};
Geo geo(bool bf16, int64_t d) {
  const int64_t vec = bf16 ? 8 : 4;
  const bool v = d % vec == 0;
  const int64_t w = v ? vec : 1, most = 8 / w;
  for (int tpr : {16, 64, 256, 512, 1024}) {
    const int64_t need = (d + tpr * w - 1) / (tpr * w);
    if (need > most) continue;
    int nv = 1;
    while (nv < need) nv *= 2;
    if (!v && nv < 4) nv = 4;
    return {tpr, nv, tpr > 256 ? tpr : 256, v};
  }
  return {0, 0, 0, false};
}

int64_t groups_of(const Geo& g) { return g.nthr / g.tpr; }
// workgroups of the backward pass: enough to fill the device four times over
int64_t bw_grid(const Geo& g, int64_t N) {
  const int64_t need = (N + groups_of(g) - 1) / groups_of(g);
  return std::min<int64_t>(need, g.nthr > 256 ? 512 : 1024);
}

template <bool BACK, int DT, int VEC, int NV, int TPR>
void go(const NormDev& a, unsigned grid, hipStream_t st) {
  constexpr int NTHR = TPR > 256 ? TPR : 256;
  if constexpr (BACK)
    k_block_norm_backward<DT, VEC, NV, TPR, NTHR><<<grid, NTHR, 0, st>>>(a);
  else
    k_block_norm<DT, VEC, NV, TPR, NTHR><<<grid, NTHR, 0, st>>>(a);
}
template <bool BACK, int DT, int VEC, int NV>
void go_tpr(const Geo& g, const NormDev& a, unsigned grid, hipStream_t st) {
  switch (g.tpr) {
    case 16: return go<BACK, DT, VEC, NV, 16>(a, grid, st);
    case 64: return go<BACK, DT, VEC, NV, 64>(a, grid, st);
    case 256: return go<BACK, DT, VEC, NV, 256>(a, grid, st);
    case 512: return go<BACK, DT, VEC, NV, 512>(a, grid, st);
    default: return go<BACK, DT, VEC, NV, 1024>(a, grid, st);
  }
}
template <bool BACK>
void go_all(bool bf16, const Geo& g, const NormDev& a, unsigned grid, hipStream_t st) {
  if (g.vec && bf16) return go_tpr<BACK, kBF16, 8, 1>(g, a, grid, st);
  if (g.vec) {
    if (g.nv == 1) return go_tpr<BACK, kF32, 4, 1>(g, a, grid, st);
    return go_tpr<BACK, kF32, 4, 2>(g, a, grid, st);
  }
  if (bf16) {
    if (g.nv == 4) return go_tpr<BACK, kBF16, 1, 4>(g, a, grid, st);
    return go_tpr<BACK, kBF16, 1, 8>(g, a, grid, st);
  }
  if (g.nv == 4) return go_tpr<BACK, kF32, 1, 4>(g, a, grid, st);
  return go_tpr<BACK, kF32, 1, 8>(g, a, grid, st);
}

}  // namespace

size_t block_norm_backward_workspace(bool bf16, int64_t N, int64_t d) {
  return size_t(3) * std::max<int64_t>(1, bw_grid(geo(bf16, d), N)) * d * 4;
}

void launch_block_norm(const BlockNormArgs& a) {
  const Geo g = geo(a.bf16, a.d);
  NormDev n{};
  n.h = a.h, n.gate = a.gate, n.x = a.x;
  n.o0 = a.r_out, n.o1 = a.n_out;
  n.w_post = a.w_post, n.w_pre = a.w_pre, n.alpha = a.alpha;
  n.N = a.N, n.d = int(a.d), n.act = a.act, n.eps = a.eps;
  go_all<false>(a.bf16, g, n, unsigned((a.N + groups_of(g) - 1) / groups_of(g)), a.stream);
}

void launch_block_norm_backward(const BlockNormArgs& a) {
  const Geo g = geo(a.bf16, a.d);
  const int64_t G = bw_grid(g, a.N);
  NormDev n{};
  n.h = a.h, n.gate = a.gate, n.x = a.x, n.dr = a.dr, n.dn = a.dn;
  n.o0 = a.dh, n.o1 = a.dgate, n.o2 = a.dx;
  n.w_post = a.w_post, n.w_pre = a.w_pre, n.alpha = a.alpha;
  n.part = reinterpret_cast<float*>(a.ws);
  n.N = a.N, n.d = int(a.d), n.act = a.act, n.eps = a.eps;
  if (G > 0) go_all<true>(a.bf16, g, n, unsigned(G), a.stream);
  if (a.dw_post || a.dw_pre || a.dalpha) {
    const dim3 grid(unsigned((a.d + 63) / 64), 3);
    k_block_norm_weights<<<grid, 1024, 0, a.stream>>>(n.part, int(G), int(a.d), a.dw_post, a.dw_pre, a.dalpha);
  }
}

}  // namespace prn
