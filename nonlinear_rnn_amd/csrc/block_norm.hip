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

// VEC elements (16 bytes, or one where a row is shorter) at any element's
// address: rows of odd widths start anywhere, and global memory takes
// unaligned vector accesses.
template <int DT, int VEC>
struct __attribute__((packed, aligned(sizeof(typename Storage<DT>::T)))) Vec {
  typename Storage<DT>::T v[VEC];
};

struct NormDev {
  const void *h, *gate, *x, *dr, *dn;
  void *o0, *o1, *o2;   // forward: r, n; backward: dh, dgate, dx
  const float *w_post, *w_pre, *alpha;
  float* part;          // backward: the workgroups' weight-gradient sums, 3 x G x d
  int64_t N;
  int d, act;
  float eps;
  bool in_place;        // forward: r is written over h or x
};

// A lane's channels: chunk v of VEC channels starts at (v TPR + lane) VEC.
// TAIL (d no multiple of VEC): the row's last chunk is moved back to end with
// the row; the channels it then shares with the chunk before it get the same
// values from both lanes, and count in sums only once (`fresh`).
template <int DT, int VEC, int NV, int TPR, bool TAIL>
struct Row {
  static constexpr int E = VEC * NV;
  using T = typename Storage<DT>::T;
  struct Raw {
    Vec<DT, VEC> v[NV];
  };
  int lane, d;
  __device__ __forceinline__ int chunk(int v) const { return (v * TPR + lane) * VEC; }
  __device__ __forceinline__ bool in(int v) const { return chunk(v) < d; }
  __device__ __forceinline__ int at(int v) const { return TAIL ? min(chunk(v), d - VEC) : chunk(v); }
  // does element e of chunk v count in sums?
  __device__ __forceinline__ bool fresh(int v, int e) const { return !TAIL || chunk(v) <= d - VEC || at(v) + e >= chunk(v); }
  __device__ __forceinline__ void fetch(const void* p, int64_t row, Raw& o) const {
    const T* q = static_cast<const T*>(p) + row * d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (in(v)) {
        o.v[v] = *reinterpret_cast<const Vec<DT, VEC>*>(q + at(v));
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o.v[v].v[e] = T(0);
      }
    }
  }
  __device__ __forceinline__ void unpack(const Raw& q, float* o) const {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < VEC; ++e) o[v * VEC + e] = Storage<DT>::load(&q.v[v].v[e]);
  }
  __device__ __forceinline__ void load(const void* p, int64_t row, float* o) const {
    Raw q;
    fetch(p, row, q);
    unpack(q, o);
  }
  __device__ __forceinline__ void store(void* p, int64_t row, const float* o) const {
    T* q = static_cast<T*>(p) + row * d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (in(v)) {
        Vec<DT, VEC> t;
#pragma unroll
        for (int e = 0; e < VEC; ++e) t.v[e] = Storage<DT>::pack(o[v * VEC + e]);
        *reinterpret_cast<Vec<DT, VEC>*>(q + at(v)) = t;
      }
    }
  }
  // fp32 weights of the lane's channels; absent: ones
  __device__ __forceinline__ void weights(const float* p, float* o) const {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < VEC; ++e) o[v * VEC + e] = (p && in(v)) ? p[at(v) + e] : 1.0f;
  }
  // sums of squares and the like: adds f(i) for every element that counts
  template <class F>
  __device__ __forceinline__ float sum(F f) const {
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += fresh(v, e) ? f(v * VEC + e) : 0.0f;
    return s;
  }
};

// 1 / sqrt(v); v_rsq_f32 takes a value below 2^-126 for zero
__device__ __forceinline__ float inverse_root(float v) {
  const bool tiny = v < 0x1p-96f;
  return __builtin_amdgcn_rsqf(tiny ? v * 0x1p96f : v) * (tiny ? 0x1p48f : 1.0f);
}

__device__ __forceinline__ float sig(float g) { return rcp(1.0f + ex2(kSigScale * g)); }

template <int DT, int VEC, int NV, int TPR, int NTHR, bool TAIL>
__global__ void __launch_bounds__(NTHR) k_block_norm(NormDev a) {
  using R = Row<DT, VEC, NV, TPR, TAIL>;
  using Raw = typename R::Raw;
  constexpr int E = R::E, GROUPS = NTHR / TPR;
  static_assert(GROUPS == 1 || TPR <= 64, "a row of several waves is its workgroup's only one (barriers)");
  __shared__ float red[2][1][TPR > 64 ? TPR / 64 : 1];
  const R row{static_cast<int>(threadIdx.x) % TPR, a.d};
  RowSum<TPR, 1> total{red};
  const float inv_d = 1.0f / static_cast<float>(a.d);
  float w_post[E], w_pre[E], alpha[E];
  row.weights(a.w_post, w_post);
  row.weights(a.w_pre, w_pre);
  row.weights(a.alpha, alpha);
  const int64_t step = static_cast<int64_t>(gridDim.x) * GROUPS;
  // the next row's operands are in flight while a row is worked on
  Raw rh, rg, rx;
  auto fetch = [&](int64_t n) {
    row.fetch(a.h, n, rh);
    if (a.gate) row.fetch(a.gate, n, rg);
    if (a.x) row.fetch(a.x, n, rx);
  };
  int64_t n = static_cast<int64_t>(blockIdx.x) * GROUPS + threadIdx.x / TPR;
  if (n < a.N) fetch(n);
  for (; n < a.N; n += step) {
    float h[E], g[E], x[E];
    row.unpack(rh, h);
    if (a.gate) row.unpack(rg, g);
    if (a.x) row.unpack(rx, x);
    if (n + step < a.N) fetch(n + step);
    if (a.w_post) {
      float s = row.sum([&](int i) { return h[i] * h[i]; });
      total(&s);
      const float rstd = inverse_root(fmaf(s, inv_d, a.eps));
#pragma unroll
      for (int e = 0; e < E; ++e) h[e] *= rstd * w_post[e];
    }
    if (a.gate) {
#pragma unroll
      for (int e = 0; e < E; ++e) h[e] *= a.act == 0 ? g[e] * sig(g[e]) : sig(g[e]);
    }
    if (a.x) {
#pragma unroll
      for (int e = 0; e < E; ++e) h[e] = fmaf(alpha[e], h[e], x[e]);
    } else if (a.alpha) {
#pragma unroll
      for (int e = 0; e < E; ++e) h[e] *= alpha[e];
    }
    // r over h or x: a moved-back last chunk reads channels that another wave
    // of the row writes, so every wave has read the row before one writes it
    // (behind the first norm's sum they have; n's stores are behind the second's)
    if constexpr (TAIL && TPR > 64) {
      if (a.in_place && !a.w_post) __syncthreads();
    }
    if (a.o0) row.store(a.o0, n, h);
    if (a.w_pre) {
      float s = row.sum([&](int i) { return h[i] * h[i]; });
      total(&s);
      const float rstd = inverse_root(fmaf(s, inv_d, a.eps));
#pragma unroll
      for (int e = 0; e < E; ++e) h[e] *= rstd * w_pre[e];
      row.store(a.o1, n, h);
    }
  }
}

template <int DT, int VEC, int NV, int TPR, int NTHR, bool TAIL>
__global__ void __launch_bounds__(NTHR) k_block_norm_backward(NormDev a) {
  using R = Row<DT, VEC, NV, TPR, TAIL>;
  using Raw = typename R::Raw;
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
  // the next row's operands are in flight while a row is worked on
  Raw rh, rg, rx, rr, rn;
  auto fetch = [&](int64_t n) {
    row.fetch(a.h, n, rh);
    if (a.gate) row.fetch(a.gate, n, rg);
    if (a.x) row.fetch(a.x, n, rx);
    if (a.dr) row.fetch(a.dr, n, rr);
    if (a.w_pre) row.fetch(a.dn, n, rn);
  };
  constexpr bool AHEAD = NTHR < 1024;   // 128 registers a lane have no room for them
  int64_t n = static_cast<int64_t>(blockIdx.x) * GROUPS + threadIdx.x / TPR;
  if (AHEAD && n < a.N) fetch(n);
  for (; n < a.N; n += step) {
    if (!AHEAD) fetch(n);
    float h[E], g[E], x[E], dr[E], dn[E];
    row.unpack(rh, h);
    if (a.gate) row.unpack(rg, g);
    if (a.x) row.unpack(rx, x);
    if (a.w_pre) row.unpack(rn, dn);
    if (a.dr) {
      row.unpack(rr, dr);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) dr[e] = 0.0f;
    }
    if (AHEAD && n + step < a.N) fetch(n + step);
    float rstd_h = 1.0f;
    if (a.w_post) {
      float s = row.sum([&](int i) { return h[i] * h[i]; });
      total(&s);
      rstd_h = inverse_root(fmaf(s, inv_d, a.eps));
#pragma unroll
      for (int e = 0; e < E; ++e) h[e] *= rstd_h;
    }
    // h is hn from here on; f = act(gate), g = act'(gate), v = hn w_post f
    float f[E], v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      f[e] = 1.0f;
      if (a.gate) {
        const float sg = sig(g[e]);
        f[e] = a.act == 0 ? g[e] * sg : sg;
        g[e] = a.act == 0 ? sg * fmaf(g[e], 1.0f - sg, 1.0f) : sg * (1.0f - sg);
      }
      v[e] = h[e] * w_post[e] * f[e];
    }
    if (a.w_pre) {
      float r[E], s[2];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        r[e] = a.x ? fmaf(alpha[e], v[e], x[e]) : alpha[e] * v[e];
      }
      s[0] = row.sum([&](int i) { return r[i] * r[i]; });
      s[1] = row.sum([&](int i) { return dn[i] * w_pre[i] * r[i]; });
      total2(s);
      const float rstd = inverse_root(fmaf(s[0], inv_d, a.eps));
      const float mean = s[1] * rstd * inv_d;   // mean(q rn)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float rn_ = r[e] * rstd;
        s_pre[e] = fmaf(dn[e], rn_, s_pre[e]);
        dr[e] = fmaf(rstd, fmaf(dn[e], w_pre[e], -rn_ * mean), dr[e]);
      }
    }
    if (a.o2) row.store(a.o2, n, dr);
    float dg[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      s_alpha[e] = fmaf(dr[e], v[e], s_alpha[e]);
      const float dv = dr[e] * alpha[e];
      if (a.gate) dg[e] = dv * h[e] * w_post[e] * g[e];
      const float du = dv * f[e];
      s_post[e] = fmaf(du, h[e], s_post[e]);
      dr[e] = du * w_post[e];
    }
    if (a.o1) row.store(a.o1, n, dg);
    if (a.w_post) {
      float s = row.sum([&](int i) { return dr[i] * h[i]; });
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
          if (row.in(v) && row.fresh(v, e))
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
          if (row.in(v) && row.fresh(v, e)) out[row.at(v) + e] = k == 0 ? s_post[i] : k == 1 ? s_pre[i] : s_alpha[i];
        }
    }
  }
}

// out_k[c] = the sum over the G workgroups' partials, for 16 channels: 64
// groups of 16 lanes take every 64th partial in order, their sums are added in
// a fixed order.  (64 channels a workgroup fill too few CUs: at d = 1001 and
// 1024 partials 5.7 us where this takes 5.0.)
constexpr int kWeightCols = 16;
__global__ void __launch_bounds__(1024) k_block_norm_weights(const float* __restrict__ part, int G, int d,
                                                             float* o0, float* o1, float* o2) {
  __shared__ float hand[16][kWeightCols];
  const int k = blockIdx.y, col = threadIdx.x % kWeightCols, c = blockIdx.x * kWeightCols + col;
  float* const out = k == 0 ? o0 : k == 1 ? o1 : o2;
  if (!out) return;
  const float* p = part + static_cast<int64_t>(k) * G * d;
  float s = 0.0f;
  if (c < d) {
#pragma unroll 8
    for (int g = threadIdx.x / kWeightCols; g < G; g += 1024 / kWeightCols) s += p[static_cast<int64_t>(g) * d + c];
  }
  s += __shfl_xor(s, 16, 64);
  s += __shfl_xor(s, 32, 64);
  if ((threadIdx.x & 63) < kWeightCols) hand[threadIdx.x >> 6][col] = s;
  __syncthreads();
  if (threadIdx.x < kWeightCols && c < d) {
    s = hand[0][col];
#pragma unroll
    for (int q = 1; q < 16; ++q) s += hand[q][col];
    out[c] = s;
  }
}

// Lanes per row, chunks per lane, workgroup: at most 8 channels a lane (16
// take the backward pass past 256 registers).  Rows shorter than 16 bytes go
// by single elements, rows of no multiple of 16 bytes with a moved-back tail.
struct Geo {
  int tpr, nv, nthr;
  bool vec, tail;
};
Geo geo(bool bf16, int64_t d) {
  const int64_t vec = bf16 ? 8 : 4;
  const bool v = d >= vec;
  const int64_t w = v ? vec : 1, most = v ? 8 / vec : 1;
  for (int tpr : {16, 64, 128, 256, 512, 1024}) {
    const int64_t need = (d + tpr * w - 1) / (tpr * w);
    if (need > most) continue;
    return {tpr, int(need), tpr > 64 ? tpr : 256, v, v && d % vec != 0};
  }
  return {0, 0, 0, false, false};
}

int64_t groups_of(const Geo& g) { return g.nthr / g.tpr; }
// Workgroups: 2 waves a SIMD at 8 channels a lane, 4 at 4 (what the backward
// kernels' registers allow; more bring nothing forward either), or one per
// group of rows where those are fewer.  Measured at 262144 x 512 bf16 with
// every part: 2, 4, 8 waves a SIMD forward 233, 262, 273 us; one workgroup per
// four rows, without the row ahead, 311 us; backward 2 or 4 waves 401, 425 us,
// without the row ahead 610 us.
int64_t grid_of(const Geo& g, bool bf16, int64_t N) {
  const int64_t need = (N + groups_of(g) - 1) / groups_of(g);
  const int64_t waves = 256 * 4 * ((bf16 || g.nv == 2) ? 2 : 4);
  return std::min<int64_t>(need, std::max<int64_t>(256, waves / (g.nthr / 64)));
}

template <bool BACK, int DT, int VEC, int NV, int TPR, bool TAIL>
void go(const NormDev& a, unsigned grid, hipStream_t st) {
  constexpr int NTHR = TPR > 64 ? TPR : 256;
  if constexpr (BACK)
    k_block_norm_backward<DT, VEC, NV, TPR, NTHR, TAIL><<<grid, NTHR, 0, st>>>(a);
  else
    k_block_norm<DT, VEC, NV, TPR, NTHR, TAIL><<<grid, NTHR, 0, st>>>(a);
}
template <bool BACK, int DT, int VEC, int NV, bool TAIL>
void go_tpr(const Geo& g, const NormDev& a, unsigned grid, hipStream_t st) {
  switch (g.tpr) {
    case 16: return go<BACK, DT, VEC, NV, 16, TAIL>(a, grid, st);
    case 64: return go<BACK, DT, VEC, NV, 64, TAIL>(a, grid, st);
    case 128: return go<BACK, DT, VEC, NV, 128, TAIL>(a, grid, st);
    case 256: return go<BACK, DT, VEC, NV, 256, TAIL>(a, grid, st);
    case 512: return go<BACK, DT, VEC, NV, 512, TAIL>(a, grid, st);
    default: return go<BACK, DT, VEC, NV, 1024, TAIL>(a, grid, st);
  }
}
template <bool BACK, int DT>
void go_vec(const Geo& g, const NormDev& a, unsigned grid, hipStream_t st) {
  constexpr int VEC = 16 / sizeof(typename Storage<DT>::T);
  if (!g.vec) return go<BACK, DT, 1, 1, 16, false>(a, grid, st);
  if (g.nv == 1) return g.tail ? go_tpr<BACK, DT, VEC, 1, true>(g, a, grid, st) : go_tpr<BACK, DT, VEC, 1, false>(g, a, grid, st);
  if constexpr (VEC == 4)
    return g.tail ? go_tpr<BACK, DT, VEC, 2, true>(g, a, grid, st) : go_tpr<BACK, DT, VEC, 2, false>(g, a, grid, st);
}
template <bool BACK>
void go_all(bool bf16, const Geo& g, const NormDev& a, unsigned grid, hipStream_t st) {
  if (bf16) go_vec<BACK, kBF16>(g, a, grid, st); else go_vec<BACK, kF32>(g, a, grid, st);
}

}  // namespace

size_t block_norm_backward_workspace(bool bf16, int64_t N, int64_t d) {
  return size_t(3) * std::max<int64_t>(1, grid_of(geo(bf16, d), bf16, N)) * d * 4;
}

void launch_block_norm(const BlockNormArgs& a) {
  const Geo g = geo(a.bf16, a.d);
  NormDev n{};
  n.h = a.h, n.gate = a.gate, n.x = a.x;
  n.o0 = a.r_out, n.o1 = a.n_out;
  n.w_post = a.w_post, n.w_pre = a.w_pre, n.alpha = a.alpha;
  n.N = a.N, n.d = int(a.d), n.act = a.act, n.eps = a.eps;
  n.in_place = a.r_out && (a.r_out == a.h || a.r_out == a.x);
  go_all<false>(a.bf16, g, n, unsigned(grid_of(g, a.bf16, a.N)), a.stream);
}

void launch_block_norm_backward(const BlockNormArgs& a) {
  const Geo g = geo(a.bf16, a.d);
  const int64_t G = grid_of(g, a.bf16, a.N);
  NormDev n{};
  n.h = a.h, n.gate = a.gate, n.x = a.x, n.dr = a.dr, n.dn = a.dn;
  n.o0 = a.dh, n.o1 = a.dgate, n.o2 = a.dx;
  n.w_post = a.w_post, n.w_pre = a.w_pre, n.alpha = a.alpha;
  n.part = reinterpret_cast<float*>(a.ws);
  n.N = a.N, n.d = int(a.d), n.act = a.act, n.eps = a.eps;
  if (G > 0) go_all<true>(a.bf16, g, n, unsigned(G), a.stream);
  if (a.dw_post || a.dw_pre || a.dalpha) {
    const dim3 grid(unsigned((a.d + kWeightCols - 1) / kWeightCols), 3);
    k_block_norm_weights<<<grid, 1024, 0, a.stream>>>(n.part, int(G), int(a.d), a.dw_post, a.dw_pre, a.dalpha);
  }
}

}  // namespace prn
