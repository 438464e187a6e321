// Gated linear recurrence over time, and its gradients.
//
//   h_t = f_t h_{t-1} + u_t      f = s(x_f)      u = (1 - f) v  (G = 2)   or  s(x_i) v  (G = 3)
//   lam_t = dH_t + f_{t+1} lam_{t+1}              (dlast added at a sequence's last step)
//   dx_f = lam (h_{t-1} - v) f (1 - f)  (G = 2)   or  lam h_{t-1} f (1 - f)
//   dx_i = lam v i (1 - i),  dv = lam i           (i = 1 - f for G = 2),   dh0 = f lam at the head
//
// Every step is an affine map of the state, per channel, so a stretch of time
// is one too: (a, b) with h_out = a h_in + b.  Backwards, with m_t the gradient
// that arrives at h_t from the steps after it, m_{t-1} = f_t (dH_t + m_t) is
// another.  A chain is one row and 64 V channels (a lane has V of them).
//
//   k_scan_map    where there are fewer chains than the device takes, time is
//                 cut in ranges and the map of each range is taken first
//   k_scan_walk   a workgroup walks its range in chunks of kWaves x kSteps
//                 steps, kSteps a wave: every wave takes the map of its steps
//                 (held in registers), the maps meet in LDS, and each wave
//                 walks its steps from its own carry.  The next chunk's loads
//                 are in flight meanwhile.  The range's own carry is the maps
//                 of the ranges before it, applied to h0.
//
// Nothing waits for another workgroup, no memory has to be cleared first, and
// every sum has a fixed order.  The walk reads and writes each value once; the
// maps read the gates (and v or dH) once more, of which up to 256 MB come from
// the memory-side cache.  Bound: memory traffic.
//
// The gradient needs h_{t-1}: it is formed again from x and the stored H of
// the step before a chunk (so only one step in kWaves kSteps sees H's
// rounding), which reads a value per step less than stored states would.
//
// A sequence's first step in a pack cuts the map: h_in does not count, whatever
// it is (a NaN of the sequence before stays there).  Since a >= 0 otherwise,
// a = -0 says so, and stays -0 in every product with what comes after.
#include "gated_scan.h"

#include <algorithm>
#include <type_traits>

#include "gated_cell.h"
#include "grid_rows.h"
#include "prn_device.h"

namespace prn {
namespace {

constexpr int kWaves = 8, kSteps = 8;    // of a workgroup, of a wave and chunk
constexpr int kChunk = kWaves * kSteps;
constexpr float kCut = -0.0f;

__device__ __forceinline__ bool is_cut(float a) { return __float_as_uint(a) == 0x80000000u; }

struct Map {
  float a, b;
};
__device__ __forceinline__ float through(const Map& m, float h) { return is_cut(m.a) ? m.b : fmaf(m.a, h, m.b); }
// first m1, then m2
__device__ __forceinline__ Map then(const Map& m1, const Map& m2) {
  return {is_cut(m2.a) ? kCut : m2.a * m1.a, through(m2, m1.b)};
}

// a barrier for what waves hand over in LDS; global loads stay in flight
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// V neighbouring channels at p (aligned to them)
template <int DT, int V>
struct Chans {
  using T = typename Storage<DT>::T;
  T v[V];
  __device__ __forceinline__ void load(const T* p) { __builtin_memcpy(v, __builtin_assume_aligned(p, V * sizeof(T)), sizeof(v)); }
  __device__ __forceinline__ void store(T* p) const { __builtin_memcpy(__builtin_assume_aligned(p, V * sizeof(T)), v, sizeof(v)); }
  __device__ __forceinline__ float at(int c) const { return Storage<DT>::load(&v[c]); }
  __device__ __forceinline__ void set(int c, float x) { v[c] = Storage<DT>::pack(x); }
};

// Where the sequences of a pack begin and end among a wave's steps: bit j of
// head / tail, and the sequence of step j.
struct Cuts {
  uint32_t head, tail;
  int32_t seg[kSteps];
  __device__ __forceinline__ void find(const int32_t* cu, int64_t n_seqs, int64_t t0, int n, int64_t T) {
    head = tail = 0;
    if (n <= 0) return;
    SegTracker s;
    s.init_wave(cu, n_seqs, 0, t0);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      if (j < n) {
        if (s.at(t0 + j)) head |= 1u << j;
        if (s.last(t0 + j, T)) tail |= 1u << j;
        seg[j] = static_cast<int32_t>(s.seg);
      }
    }
  }
};

// A workgroup's place: chain (row, channel tile) and range of time.
template <int V>
struct Place {
  int lane, wave;
  int64_t row, chain, c0;   // c0: this lane's first channel, kept in range
  bool live;                // has this lane channels of its own?
  int64_t range, t0, t1;
  bool there;               // is this workgroup one of the launch's (rows_of_blocks)?
  __device__ __forceinline__ Place(int64_t B, int64_t d, int64_t T, int ranges, int64_t per) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tiles = (d + 64 * V - 1) / (64 * V), b = block_in_rows();
    there = b < B * tiles * ranges;
    chain = b / ranges;
    range = b - chain * ranges;
    row = chain / tiles;
    c0 = (chain - row * tiles) * 64 * V + lane * V;
    live = c0 < d;
    if (!live) c0 = d - V;
    t0 = range * per;
    t1 = imin(t0 + per, T);
  }
};

// the maps of a chain's ranges, in the order they are walked: [chain][range][a, b][V][64]
template <int V>
__device__ __forceinline__ float* map_at(float* maps, int64_t chain, int ranges, int64_t range) {
  return maps + ((chain * ranges + range) * 2 * V) * 64;
}

// The map of ranges [0, n) of a chain: wave w joins its share of them, and the
// shares meet in `part`.  Every wave has it after the call.
template <int V>
__device__ __forceinline__ void maps_before(const float* maps, int64_t chain, int ranges, int n, int lane, int wave,
                                            Map (*part)[V][64], Map (&out)[V]) {
  constexpr int kAhead = 8;
  const int per = (n + kWaves - 1) / kWaves, i0 = min(wave * per, n), i1 = min(i0 + per, n);
  Map m[V];
#pragma unroll
  for (int c = 0; c < V; ++c) m[c] = {1.0f, 0.0f};
  for (int i = i0; i < i1; i += kAhead) {
    Map q[kAhead][V];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const float* p = map_at<V>(const_cast<float*>(maps), chain, ranges, min(i + k, i1 - 1)) + lane;
#pragma unroll
      for (int c = 0; c < V; ++c) q[k][c] = {p[c * 64], p[(V + c) * 64]};
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + k < i1) {
#pragma unroll
        for (int c = 0; c < V; ++c) m[c] = then(m[c], q[k][c]);
      }
  }
#pragma unroll
  for (int c = 0; c < V; ++c) part[wave][c][lane] = m[c];
  lds_barrier();
#pragma unroll
  for (int c = 0; c < V; ++c) out[c] = part[0][c][lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w)
#pragma unroll
    for (int c = 0; c < V; ++c) out[c] = then(out[c], part[w][c][lane]);
  lds_barrier();   // part is free again
}

// --------------------------------------------------------------- maps ----

// A range's map: wave w takes the w-th eighth of it.  BACK: of the gradient,
// from the last step to the first, the maps stored in that order.
template <int DT, int G, int V, bool RAGGED, bool BACK>
__global__ void __launch_bounds__(64 * kWaves) k_scan_map(const typename Storage<DT>::T* __restrict__ x,
                                                          const typename Storage<DT>::T* __restrict__ h0,
                                                          const typename Storage<DT>::T* __restrict__ dH,
                                                          const typename Storage<DT>::T* __restrict__ dlast,
                                                          const int32_t* __restrict__ cu, int64_t n_seqs, int64_t B,
                                                          int64_t T, int64_t d, int ranges, int64_t per, float* __restrict__ maps) {
  using C = Chans<DT, V>;
  __shared__ Map part[kWaves][V][64];
  const Place<V> at(B, d, T, ranges, per);
  if (!at.there) return;
  const int64_t share = (per + kWaves - 1) / kWaves;
  const int64_t s0 = imin(at.t0 + at.wave * share, at.t1), s1 = imin(s0 + share, at.t1);
  constexpr int R = BACK ? 2 : G;   // values read of a step: f and dH, or all of x
  auto read = [&](int64_t t, C (&q)[R]) {
    const typename Storage<DT>::T* p = x + ((at.row * T + t) * G) * d + at.c0;
    if constexpr (BACK) {
      q[0].load(p);
      q[1].load(dH + (at.row * T + t) * d + at.c0);
    } else {
#pragma unroll
      for (int g = 0; g < G; ++g) q[g].load(p + g * d);
    }
  };
  Map m[V];
#pragma unroll
  for (int c = 0; c < V; ++c) m[c] = {1.0f, 0.0f};
  const int blocks = static_cast<int>((s1 - s0 + kSteps - 1) / kSteps);
  // step j of block k, in the order of the walk (a step past the end: the last one, not used)
  auto step_at = [&](int k, int j) {
    const int64_t i = static_cast<int64_t>(k) * kSteps + j;
    return BACK ? imax(s1 - 1 - i, s0) : imin(s0 + i, s1 - 1);
  };
  C q[2][kSteps][R];
  auto load_block = [&](int k, C (&to)[kSteps][R]) {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) read(step_at(k, j), to[j]);
  };
  auto use_block = [&](int k, const C (&v)[kSteps][R]) {
    const int n = static_cast<int>(imin(kSteps, s1 - s0 - static_cast<int64_t>(k) * kSteps));
    Cuts cut;
    const int64_t first = BACK ? step_at(k, n - 1) : step_at(k, 0);
    if constexpr (RAGGED) cut.find(cu, n_seqs, first, n, T);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      if (j >= n) break;
      const int bit = BACK ? n - 1 - j : j;
      const bool here = RAGGED && (((BACK ? cut.tail : cut.head) >> bit) & 1);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const Gate f = gate_of(v[j][0].at(c));
        Map s;
        if constexpr (BACK) {
          float g = v[j][1].at(c);
          if (RAGGED ? here : step_at(k, j) == T - 1) {
            if (dlast) g += Storage<DT>::load(dlast + (RAGGED ? cut.seg[bit] : at.row) * d + at.c0 + c);
          }
          s = {here ? kCut : f.on, f.on * g};
        } else {
          s = {f.on, (G == 2 ? f.off : gate_of(v[j][1].at(c)).on) * v[j][R - 1].at(c)};
          if (here) {
            if (h0) s.b = fmaf(s.a, Storage<DT>::load(h0 + static_cast<int64_t>(cut.seg[bit]) * d + at.c0 + c), s.b);
            s.a = kCut;
          }
        }
        m[c] = then(m[c], s);
      }
    }
  };
  if (blocks > 0) load_block(0, q[0]);
  for (int k = 0; k < blocks; k += 2) {
    if (k + 1 < blocks) load_block(k + 1, q[1]);
    use_block(k, q[0]);
    if (k + 1 >= blocks) break;
    if (k + 2 < blocks) load_block(k + 2, q[0]);
    use_block(k + 1, q[1]);
  }
#pragma unroll
  for (int c = 0; c < V; ++c) part[at.wave][c][at.lane] = m[c];
  lds_barrier();
  if (at.wave != 0) return;
#pragma unroll
  for (int c = 0; c < V; ++c) {
    Map t = part[BACK ? kWaves - 1 : 0][c][at.lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) t = then(t, part[BACK ? kWaves - 1 - w : w][c][at.lane]);
    float* p = map_at<V>(maps, at.chain, ranges, BACK ? ranges - 1 - at.range : at.range) + at.lane;
    p[c * 64] = t.a;
    p[(V + c) * 64] = t.b;
  }
}

// ------------------------------------------------------------- forward ----

template <int DT, int G, int V, bool RAGGED>
__global__ void __launch_bounds__(64 * kWaves) k_scan_walk(const typename Storage<DT>::T* __restrict__ x,
                                                           const typename Storage<DT>::T* __restrict__ h0,
                                                           const int32_t* __restrict__ cu, int64_t n_seqs, int64_t B,
                                                           int64_t T, int64_t d, int ranges, int64_t per,
                                                           const float* __restrict__ maps,
                                                           typename Storage<DT>::T* __restrict__ H,
                                                           typename Storage<DT>::T* __restrict__ last) {
  using C = Chans<DT, V>;
  __shared__ Map part[2][kWaves][V][64];
  const Place<V> at(B, d, T, ranges, per);
  if (!at.there) return;
  const typename Storage<DT>::T* const xr = x + at.row * T * G * d + at.c0;
  typename Storage<DT>::T* const Hr = H + at.row * T * d + at.c0;
  const int chunks = static_cast<int>((at.t1 - at.t0 + kChunk - 1) / kChunk);
  C q[2][kSteps][G];
  auto load_chunk = [&](int k, C (&to)[kSteps][G]) {
    const int64_t s0 = at.t0 + static_cast<int64_t>(k) * kChunk + at.wave * kSteps;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int64_t t = imin(s0 + j, at.t1 - 1);
#pragma unroll
      for (int g = 0; g < G; ++g) to[j][g].load(xr + (t * G + g) * d);
    }
  };
  load_chunk(0, q[0]);
  float h[V];   // the state before the chunk
#pragma unroll
  for (int c = 0; c < V; ++c) h[c] = !RAGGED && h0 ? Storage<DT>::load(h0 + at.row * d + at.c0 + c) : 0.0f;
  if (at.range > 0) {
    Map m[V];
    maps_before<V>(maps, at.chain, ranges, static_cast<int>(at.range), at.lane, at.wave, part[0], m);
#pragma unroll
    for (int c = 0; c < V; ++c) h[c] = through(m[c], h[c]);
  }
  auto use_chunk = [&](int k, const C (&v)[kSteps][G]) {
    const int64_t s0 = at.t0 + static_cast<int64_t>(k) * kChunk + at.wave * kSteps;
    const int n = static_cast<int>(imax(imin(kSteps, at.t1 - s0), 0));
    Cuts cut;
    if constexpr (RAGGED) cut.find(cu, n_seqs, s0, n, T);
    Map s[kSteps][V], m[V];
#pragma unroll
    for (int c = 0; c < V; ++c) m[c] = {1.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const bool here = RAGGED && j < n && ((cut.head >> j) & 1);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const Gate f = gate_of(v[j][0].at(c));
        s[j][c] = {f.on, (G == 2 ? f.off : gate_of(v[j][1].at(c)).on) * v[j][G - 1].at(c)};
        if (here) {
          if (h0) s[j][c].b = fmaf(f.on, Storage<DT>::load(h0 + static_cast<int64_t>(cut.seg[j]) * d + at.c0 + c), s[j][c].b);
          s[j][c].a = kCut;
        }
        if (j < n) m[c] = then(m[c], s[j][c]);
      }
    }
    Map(*const p)[V][64] = part[k & 1];
#pragma unroll
    for (int c = 0; c < V; ++c) p[at.wave][c][at.lane] = m[c];
    lds_barrier();
    float mine[V];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        if (w == at.wave) mine[c] = h[c];
        h[c] = through(p[w][c][at.lane], h[c]);
      }
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      if (j >= n) break;
      C o;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        mine[c] = through(s[j][c], mine[c]);
        o.set(c, mine[c]);
      }
      if (at.live) {
        o.store(Hr + (s0 + j) * d);
        if (last && (RAGGED ? (cut.tail >> j) & 1 : s0 + j == T - 1))
          o.store(last + (RAGGED ? cut.seg[j] : at.row) * d + at.c0);
      }
    }
  };
  for (int k = 0; k < chunks; k += 2) {
    if (k + 1 < chunks) load_chunk(k + 1, q[1]);
    use_chunk(k, q[0]);
    if (k + 1 >= chunks) break;
    if (k + 2 < chunks) load_chunk(k + 2, q[0]);
    use_chunk(k + 1, q[1]);
  }
}

// ------------------------------------------------------------ backward ----

// what a step of the backward reads
template <int DT, int G, int V>
struct BackStep {
  Chans<DT, V> x[G], g;
};

template <int DT, int G, int V, bool RAGGED>
__global__ void __launch_bounds__(64 * kWaves) k_scan_walk_back(
    const typename Storage<DT>::T* __restrict__ x, const typename Storage<DT>::T* __restrict__ h0,
    const typename Storage<DT>::T* __restrict__ H, const typename Storage<DT>::T* __restrict__ dH,
    const typename Storage<DT>::T* __restrict__ dlast, const int32_t* __restrict__ cu, int64_t n_seqs, int64_t B,
    int64_t T, int64_t d, int ranges, int64_t per, const float* __restrict__ maps, typename Storage<DT>::T* __restrict__ dx,
    typename Storage<DT>::T* __restrict__ dh0) {
  using ST = Storage<DT>;
  using C = Chans<DT, V>;
  using Step = BackStep<DT, G, V>;
  __shared__ Map fore[2][kWaves][V][64], back[2][kWaves][V][64];
  const Place<V> at(B, d, T, ranges, per);
  if (!at.there) return;
  const typename ST::T* const xr = x + at.row * T * G * d + at.c0;
  typename ST::T* const dxr = dx + at.row * T * G * d + at.c0;
  const typename ST::T* const Hr = H + at.row * T * d + at.c0;
  const typename ST::T* const gr = dH + at.row * T * d + at.c0;
  const int chunks = static_cast<int>((at.t1 - at.t0 + kChunk - 1) / kChunk);
  // chunk k from the end of the range; `start` the state before it
  Step q[2][kSteps];
  C start[2];
  auto first_of = [&](int k) { return at.t0 + static_cast<int64_t>(chunks - 1 - k) * kChunk; };
  auto load_chunk = [&](int k, Step (&to)[kSteps], C& st) {
    const int64_t f0 = first_of(k), s0 = f0 + at.wave * kSteps;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int64_t t = imin(s0 + j, at.t1 - 1);
#pragma unroll
      for (int g = 0; g < G; ++g) to[j].x[g].load(xr + (t * G + g) * d);
      to[j].g.load(gr + t * d);
    }
    if (f0 > 0) {
      st.load(Hr + (f0 - 1) * d);
    } else if (!RAGGED && h0) {
      st.load(h0 + at.row * d + at.c0);
    } else {
#pragma unroll
      for (int c = 0; c < V; ++c) st.set(c, 0.0f);
    }
  };
  load_chunk(0, q[0], start[0]);
  float mu[V];   // the gradient that arrives at the chunk's last state from the steps after it
#pragma unroll
  for (int c = 0; c < V; ++c) mu[c] = 0.0f;
  if (at.range + 1 < ranges) {
    Map m[V];
    maps_before<V>(maps, at.chain, ranges, static_cast<int>(ranges - 1 - at.range), at.lane, at.wave, back[0], m);
#pragma unroll
    for (int c = 0; c < V; ++c) mu[c] = through(m[c], 0.0f);
  }
  auto use_chunk = [&](int k, const Step (&v)[kSteps], const C& st) {
    const int64_t s0 = first_of(k) + at.wave * kSteps;
    const int n = static_cast<int>(imax(imin(kSteps, at.t1 - s0), 0));
    Cuts cut;
    if constexpr (RAGGED) cut.find(cu, n_seqs, s0, n, T);
    auto head = [&](int j) { return RAGGED && ((cut.head >> j) & 1); };
    auto tail = [&](int j) { return RAGGED && ((cut.tail >> j) & 1); };
    auto seg = [&](int j) { return RAGGED ? static_cast<int64_t>(cut.seg[j]) : at.row; };
    // the forward map of a step, and the gradient that arrives at its state from outside
    auto forward = [&](int j, int c, const Gate& f, const Gate& i) {
      Map m = {f.on, i.on * v[j].x[G - 1].at(c)};
      if (head(j)) {
        if (h0) m.b = fmaf(f.on, ST::load(h0 + seg(j) * d + at.c0 + c), m.b);
        m.a = kCut;
      }
      return m;
    };
    float g[kSteps][V];
    Gate f[kSteps][V], i[kSteps][V];
    Map mf[V], mb[V];
#pragma unroll
    for (int c = 0; c < V; ++c) mf[c] = mb[c] = {1.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        f[j][c] = gate_of(v[j].x[0].at(c));
        i[j][c] = G == 2 ? Gate{f[j][c].off, f[j][c].on} : gate_of(v[j].x[1].at(c));
        g[j][c] = v[j].g.at(c);
        if (j < n && dlast && (RAGGED ? tail(j) : s0 + j == T - 1)) g[j][c] += ST::load(dlast + seg(j) * d + at.c0 + c);
        if (j < n) mf[c] = then(mf[c], forward(j, c, f[j][c], i[j][c]));
      }
    }
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) {
      if (j >= n) continue;
#pragma unroll
      for (int c = 0; c < V; ++c) mb[c] = then(mb[c], Map{tail(j) ? kCut : f[j][c].on, f[j][c].on * g[j][c]});
    }
    Map(*const pf)[V][64] = fore[k & 1], (*const pb)[V][64] = back[k & 1];
#pragma unroll
    for (int c = 0; c < V; ++c) {
      pf[at.wave][c][at.lane] = mf[c];
      pb[at.wave][c][at.lane] = mb[c];
    }
    lds_barrier();
    float h[V], m[V];
#pragma unroll
    for (int c = 0; c < V; ++c) h[c] = st.at(c);
#pragma unroll
    for (int w = 0; w < kWaves - 1; ++w) {
      if (w >= at.wave) break;
#pragma unroll
      for (int c = 0; c < V; ++c) h[c] = through(pf[w][c][at.lane], h[c]);
    }
#pragma unroll
    for (int w = kWaves - 1; w >= 0; --w) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        if (w == at.wave) m[c] = mu[c];
        mu[c] = through(pb[w][c][at.lane], mu[c]);
      }
    }
    float prev[kSteps][V];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      if (j >= n) break;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        if (head(j)) h[c] = h0 ? ST::load(h0 + seg(j) * d + at.c0 + c) : 0.0f;
        prev[j][c] = h[c];
        h[c] = fmaf(f[j][c].on, h[c], i[j][c].on * v[j].x[G - 1].at(c));
      }
    }
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) {
      if (j >= n) continue;
      C o[G], first;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float lam = tail(j) ? g[j][c] : g[j][c] + m[c], val = v[j].x[G - 1].at(c);
        const float df = f[j][c].on * f[j][c].off;
        o[0].set(c, lam * (G == 2 ? prev[j][c] - val : prev[j][c]) * df);
        if constexpr (G == 3) o[1].set(c, lam * val * (i[j][c].on * i[j][c].off));
        o[G - 1].set(c, lam * i[j][c].on);
        m[c] = f[j][c].on * lam;
        first.set(c, m[c]);
      }
      if (at.live) {
#pragma unroll
        for (int e = 0; e < G; ++e) o[e].store(dxr + ((s0 + j) * G + e) * d);
        if (dh0 && (RAGGED ? head(j) : s0 + j == 0)) first.store(dh0 + seg(j) * d + at.c0);
      }
    }
  };
  for (int k = 0; k < chunks; k += 2) {
    if (k + 1 < chunks) load_chunk(k + 1, q[1], start[1]);
    use_chunk(k, q[0], start[0]);
    if (k + 1 >= chunks) break;
    if (k + 2 < chunks) load_chunk(k + 2, q[0], start[0]);
    use_chunk(k + 1, q[1], start[1]);
  }
}

// out[j] = in[j] (0 without in) of the sequences of a pack that have no step,
// or, without cu, of every row
template <class T>
__global__ void __launch_bounds__(256) k_scan_empty(const int32_t* __restrict__ cu, int64_t rows, int64_t d,
                                                    const T* __restrict__ in, T* __restrict__ out) {
  const int64_t i = block_in_rows() * 256 + threadIdx.x;
  if (i >= rows * d) return;
  const int64_t j = i / d;
  if (cu && cu[j + 1] > cu[j]) return;
  out[i] = in ? in[i] : T(0);
}

// ---------------------------------------------------------------- plan ----

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// workgroups that fill the device
constexpr int64_t kFill = 512;

struct Plan {
  int V;
  int64_t chains, per;
  int ranges;
  size_t total;
};
Plan plan_of(const GatedScanArgs& a) {
  Plan p{};
  if (a.T == 0) return p;
  p.V = a.bf16 && a.d % 2 == 0 ? 2 : 1;   // 4 bytes a lane where the rows allow it
  p.chains = a.B * cdiv(a.d, 64 * p.V);
  const int64_t chunks = cdiv(a.T, kChunk);
  const int64_t want = std::max<int64_t>(1, std::min(chunks, kFill / std::max<int64_t>(1, p.chains)));
  p.per = cdiv(chunks, want) * kChunk;
  p.ranges = static_cast<int>(std::max<int64_t>(1, cdiv(a.T, p.per)));
  p.total = p.ranges > 1 ? size_t(p.chains) * p.ranges * 2 * p.V * 64 * sizeof(float) : 0;
  return p;
}

template <class F>
void typed(const GatedScanArgs& a, int V, F go) {
  using std::integral_constant;
  auto ragged = [&](auto dt, auto g, auto v) {
    if (a.n_seqs > 0) go(dt, g, v, std::true_type{}); else go(dt, g, v, std::false_type{});
  };
  auto gates = [&](auto dt, auto v) {
    if (a.G == 2) ragged(dt, integral_constant<int, 2>{}, v); else ragged(dt, integral_constant<int, 3>{}, v);
  };
  if (!a.bf16)
    gates(integral_constant<int, kF32>{}, integral_constant<int, 1>{});
  else if (V == 2)
    gates(integral_constant<int, kBF16>{}, integral_constant<int, 2>{});
  else
    gates(integral_constant<int, kBF16>{}, integral_constant<int, 1>{});
}

void fill_empty(const GatedScanArgs& a, const void* in, void* out) {
  const int64_t rows = a.n_seqs > 0 ? a.n_seqs : a.B;
  const dim3 grid = rows_of_blocks(cdiv(rows * a.d, 256));
  if (a.bf16)
    k_scan_empty<uint16_t><<<grid, 256, 0, a.stream>>>(a.cu, rows, a.d, static_cast<const uint16_t*>(in), static_cast<uint16_t*>(out));
  else
    k_scan_empty<float><<<grid, 256, 0, a.stream>>>(a.cu, rows, a.d, static_cast<const float*>(in), static_cast<float*>(out));
}

}  // namespace

size_t gated_scan_workspace(const GatedScanArgs& a) { return plan_of(a).total; }
size_t gated_scan_backward_workspace(const GatedScanArgs& a) { return plan_of(a).total; }

void launch_gated_scan(const GatedScanArgs& a) {
  if (a.last && (a.n_seqs > 0 || a.T == 0)) fill_empty(a, a.h0, a.last);
  if (a.T == 0) return;
  const Plan p = plan_of(a);
  float* const maps = reinterpret_cast<float*>(a.ws);
  const dim3 grid = rows_of_blocks(p.chains * p.ranges);
  typed(a, p.V, [&](auto dt, auto g, auto v, auto ragged) {
    constexpr int DT = decltype(dt)::value, G = decltype(g)::value, V = decltype(v)::value;
    constexpr bool RAGGED = decltype(ragged)::value;
    using T = typename Storage<DT>::T;
    const T *x = static_cast<const T*>(a.xproj), *h0 = static_cast<const T*>(a.h0);
    if (p.ranges > 1)
      k_scan_map<DT, G, V, RAGGED, false><<<grid, 64 * kWaves, 0, a.stream>>>(x, h0, nullptr, nullptr, a.cu, a.n_seqs, a.B, a.T, a.d,
                                                                              p.ranges, p.per, maps);
    k_scan_walk<DT, G, V, RAGGED><<<grid, 64 * kWaves, 0, a.stream>>>(x, h0, a.cu, a.n_seqs, a.B, a.T, a.d, p.ranges, p.per, maps,
                                                                      static_cast<T*>(a.H), static_cast<T*>(a.last));
  });
}

void launch_gated_scan_backward(const GatedScanArgs& a) {
  if (a.dh0 && (a.n_seqs > 0 || a.T == 0)) fill_empty(a, a.dlast, a.dh0);
  if (a.T == 0) return;
  const Plan p = plan_of(a);
  float* const maps = reinterpret_cast<float*>(a.ws);
  const dim3 grid = rows_of_blocks(p.chains * p.ranges);
  typed(a, p.V, [&](auto dt, auto g, auto v, auto ragged) {
    constexpr int DT = decltype(dt)::value, G = decltype(g)::value, V = decltype(v)::value;
    constexpr bool RAGGED = decltype(ragged)::value;
    using T = typename Storage<DT>::T;
    const T *x = static_cast<const T*>(a.xproj), *h0 = static_cast<const T*>(a.h0), *H = static_cast<const T*>(a.H),
            *dH = static_cast<const T*>(a.dH), *dlast = static_cast<const T*>(a.dlast);
    if (p.ranges > 1)
      k_scan_map<DT, G, V, RAGGED, true><<<grid, 64 * kWaves, 0, a.stream>>>(x, h0, dH, dlast, a.cu, a.n_seqs, a.B, a.T, a.d,
                                                                             p.ranges, p.per, maps);
    k_scan_walk_back<DT, G, V, RAGGED><<<grid, 64 * kWaves, 0, a.stream>>>(x, h0, H, dH, dlast, a.cu, a.n_seqs, a.B, a.T, a.d,
                                                                           p.ranges, p.per, maps,
                                                                           static_cast<T*>(a.dxproj), static_cast<T*>(a.dh0));
  });
}

}  // namespace prn
