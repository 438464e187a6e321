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
// another.  A chain is one row and 64 V channels (a lane has V of them).  A
// workgroup has a chunk of its chain, NW waves x LS steps, LS a wave, in
// registers: every wave takes the map of its steps, the maps meet in LDS, and
// each wave walks its steps from its own carry.  Every value is read and
// written once.
//
//   k_scan_walk   where there are chains enough for the device: a workgroup
//                 walks its chain chunk after chunk, the next one's loads under
//                 way meanwhile.
//   k_scan_pass   else: chunks run side by side and get the state before them
//                 from the chunks before (look_back).
// and the same two backwards.  Bound: memory traffic (long chains: the look-back
// besides).
//
// The gradient needs h_{t-1}: it is formed again from x and the stored H of
// the step before a chunk, which reads a value per step less than stored states
// would.  That H's rounding (bf16: 2^-8 of it at most) stays in the chunk's
// states as long as the gates keep it, so dx_f = lam (h_{t-1} - v) f (1 - f) is off
// by the same lam f (1 - f) times what is left of it, with one sign over 64 to 160
// steps; stored states of H's type would each have a rounding of their own.
//
// A sequence's first step in a pack cuts the map: h_in does not count, whatever
// it is (a NaN of the sequence before stays there).  Since a >= 0 otherwise,
// a = -0 says so, and stays -0 in every product with what comes after.  Steps
// behind the last sequence get zeros.
//
// Next to the memory traffic, what counts is the arithmetic: a gate is an
// exponential and a quotient, 16 cycles of a wave each.  Rows are addressed from
// scalar registers, batches without sequences do without cuts, and whole chunks
// without bounds.
#include "gated_scan.h"

#include <algorithm>
#include <type_traits>

#include "gated_cell.h"
#include "grid_rows.h"
#include "prn_device.h"

namespace prn {
namespace {

constexpr float kCut = -0.0f;

__device__ __forceinline__ bool is_cut(float a) { return __float_as_uint(a) == 0x80000000u; }

struct Map {
  float a, b;
};
// CUTS: may the map be a cut (of a pack)?
template <bool CUTS>
__device__ __forceinline__ float through(const Map& m, float h) {
  return CUTS && is_cut(m.a) ? m.b : fmaf(m.a, h, m.b);
}
// first m1, then m2
template <bool CUTS>
__device__ __forceinline__ Map then(const Map& m1, const Map& m2) {
  return {CUTS && is_cut(m2.a) ? kCut : m2.a * m1.a, through<CUTS>(m2, m1.b)};
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
  // of a row in scalar registers, from its element off on (32-bit byte offsets, as the instructions have them)
  __device__ __forceinline__ void load(const T* row, uint32_t off) {
    load(reinterpret_cast<const T*>(reinterpret_cast<const uint8_t*>(row) + off * static_cast<uint32_t>(sizeof(T))));
  }
  __device__ __forceinline__ void store(T* row, uint32_t off) const {
    store(reinterpret_cast<T*>(reinterpret_cast<uint8_t*>(row) + off * static_cast<uint32_t>(sizeof(T))));
  }
  __device__ __forceinline__ float at(int c) const { return Storage<DT>::load(&v[c]); }
  __device__ __forceinline__ void set(const float (&x)[V]) {
    if constexpr (DT == kBF16 && V == 2) {   // one conversion of both
      typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
      const bf16x2 p{static_cast<__bf16>(x[0]), static_cast<__bf16>(x[1])};
      __builtin_memcpy(v, &p, sizeof(v));
    } else {
#pragma unroll
      for (int c = 0; c < V; ++c) v[c] = Storage<DT>::pack(x[c]);
    }
  }
};

// Where the sequences of a pack begin and end among a wave's steps: bit j of
// head / tail, and the sequence of step j.
template <int LS>
struct Cuts {
  uint32_t head, tail;
  int32_t seg[LS];
  __device__ __forceinline__ void find(const int32_t* cu, int64_t n_seqs, int64_t t0, int n, int64_t end) {
    head = tail = 0;
    if (n <= 0) return;
    SegTracker s;
    s.init_wave(cu, n_seqs, 0, t0);
#pragma unroll
    for (int j = 0; j < LS; ++j) {
      if (j < n) {
        if (s.at(t0 + j)) head |= 1u << j;
        if (s.last(t0 + j, end)) tail |= 1u << j;
        seg[j] = static_cast<int32_t>(s.seg);
      }
    }
  }
};

// the tensors of a call, and its sizes
template <int DT>
struct Tensors {
  using T = typename Storage<DT>::T;
  const T *x, *h0, *dH, *dlast;
  T *H, *last, *dx, *dh0;
  const int32_t* cu;
  int64_t n_seqs, B, T_, d;
  int64_t chains, chunks;
  // the steps of a row that belong to a sequence: a pack may end before its tensor
  template <bool RAGGED>
  __device__ __forceinline__ int64_t end() const {
    return RAGGED ? imin(imax(static_cast<int64_t>(cu[n_seqs]), 0), T_) : T_;
  }
};

// ------------------------------------------------------------ look-back ----

// Chunk c of a chain publishes its map, and, once it has the state before it,
// the state after it.  Its own carry is defined one chunk after another, E(c + 1)
// = map_c(E(c)); a chunk that finds the state after an earlier chunk p behind
// an unbroken run of published maps takes it through map_{p+1} .. map_{c-1} in
// that order: the same operations, so the bits do not depend on which state it
// found.  Workgroups take their chunks by ticket, the chunks of a chain in the
// order of its walk, so a chunk waits for chunks with smaller tickets only,
// which have started.  Every wait ends: after spin_limit polls in all that found
// a chunk without a record (looking further back is none of them) the carry is
// NaN, the error word is set, and the chunk goes on.
//
// A record's words are written and read at the device's coherence point (relaxed
// atomics of agent scope); a wave's stores have been acknowledged before it
// stores the status that announces them, and a reader loads them after it has
// the status.
struct Records {
  unsigned* ticket;
  unsigned* error;
  unsigned* status;   // [chain][chunk]: kNone, kMap, kState
  float* maps;        // [chain][chunk][a, b][V][64]
  float* states;      // [chain][chunk][V][64]
};
constexpr unsigned kNone = 0, kMap = 1, kState = 2;

__device__ __forceinline__ void put(float* p, float v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ float get(const float* p) {
  return __hip_atomic_load(const_cast<float*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void announce(unsigned* status, unsigned v, int lane) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  if (lane == 0) __hip_atomic_store(status, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// the state before chunk c > 0 of the chain whose records begin at `base`, by a whole wave
template <int V, bool CUTS>
__device__ __forceinline__ void look_back(const Records& rec, int64_t base, int64_t c, const Map (&own)[V], int lane,
                                          unsigned spin_limit, bool map_first, float (&e)[V]) {
  constexpr int kAhead = 16 / V;   // maps under way at once
  float* const mine = rec.maps + (base + c) * 2 * V * 64 + lane;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    put(mine + v * 64, own[v].a);
    put(mine + (V + v) * 64, own[v].b);
  }
  bool announced = false;
  unsigned spins = 0;
  int64_t at = c - 1;   // lane i looks at chunk at - i
  while (true) {
    if (spins >= spin_limit) {
      if (lane == 0) atomicOr(rec.error, 1u);
      if (!announced) announce(rec.status + base + c, kMap, lane);
#pragma unroll
      for (int v = 0; v < V; ++v) e[v] = __builtin_nanf("");
      return;
    }
    const int64_t j = at - lane;
    const unsigned st =
        j >= 0 ? __hip_atomic_load(rec.status + base + j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : kNone;
    const unsigned long long there = __ballot(st != kNone), state = __ballot(st == kState);
    const int run = ~there ? __builtin_ctzll(~there) : 64, first = state ? __builtin_ctzll(state) : 64;
    const bool hit = first < run;
    // (the poll's wait has covered the stores of the map)
    if ((map_first || !hit) && !announced) {
      announce(rec.status + base + c, kMap, lane);
      announced = true;
    }
    if (hit) {
      const int64_t p = at - first;
      const int n = static_cast<int>(c - 1 - p);
      const float* const from = rec.states + (base + p) * V * 64 + lane;
#pragma unroll
      for (int v = 0; v < V; ++v) e[v] = get(from + v * 64);
      for (int r = 0; r < n; r += kAhead) {
        Map m[kAhead][V];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float* const q = rec.maps + (base + p + 1 + min(r + k, n - 1)) * 2 * V * 64 + lane;
#pragma unroll
          for (int v = 0; v < V; ++v) m[k][v] = {get(q + v * 64), get(q + (V + v) * 64)};
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (r + k < n) {
#pragma unroll
            for (int v = 0; v < V; ++v) e[v] = through<CUTS>(m[k][v], e[v]);
          }
      }
      return;
    }
    if (run == 64) {   // maps only: look further back
      at -= 64;
      continue;
    }
    ++spins;
    __builtin_amdgcn_s_sleep(1);
  }
}

// A workgroup's place: its lane's channels and its wave's steps are of chain
// (row, tile of channels).
template <int V>
struct Place {
  int lane, wave;
  int64_t chain, row, tile;   // tile: its first channel
  uint32_t off;               // this lane's first channel from there, kept in range
  bool live;                  // has this lane channels of its own?
  __device__ __forceinline__ Place(int64_t d, int64_t chain_) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tiles = (d + 64 * V - 1) / (64 * V);
    chain = chain_;
    row = chain / tiles;
    tile = (chain - row * tiles) * 64 * V;
    const uint32_t left = static_cast<uint32_t>(imin(d - tile, 64 * V));   // a multiple of V
    off = lane * V;
    live = off < left;
    if (!live) off = left - V;
  }
};

// -------------------------------------------------------------- forward ----

// a wave's LS steps from s0 on
template <int DT, int G, int V, int LS, bool RAGGED>
struct Fore {
  using C = Chans<DT, V>;
  C q[LS][G];
  Map s[LS][V];
  Cuts<LS> cut;
  int64_t s0;
  int n;

  __device__ __forceinline__ void load(const Tensors<DT>& t, const Place<V>& at, int64_t first) {
    s0 = first + at.wave * LS;
    n = static_cast<int>(imax(imin(LS, t.template end<RAGGED>() - s0), 0));
    const typename C::T* const x = t.x + at.row * t.T_ * G * t.d + at.tile;
#pragma unroll
    for (int j = 0; j < LS; ++j) {
      const int64_t step = imin(s0 + j, t.T_ - 1);   // past the end: the last one, not used
#pragma unroll
      for (int g = 0; g < G; ++g) q[j][g].load(x + (step * G + g) * t.d, at.off);
    }
  }
  // the steps' maps, and the map of them all; ALL: n = LS
  template <bool ALL>
  __device__ __forceinline__ void maps_of(const Tensors<DT>& t, const Place<V>& at, Map (&m)[V]) {
#pragma unroll
    for (int j = 0; j < LS; ++j) {
      const bool here = RAGGED && (ALL || j < n) && ((cut.head >> j) & 1);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const Gate f = gate_of(q[j][0].at(c));
        s[j][c] = {f.on, (G == 2 ? f.off : gate_of(q[j][1].at(c)).on) * q[j][G - 1].at(c)};
        if (here) {   // without h0 from zero, which a NaN gate does not keep either
          const float h0 = t.h0 ? Storage<DT>::load(t.h0 + static_cast<int64_t>(cut.seg[j]) * t.d + at.tile + at.off + c) : 0.0f;
          s[j][c].b = fmaf(f.on, h0, s[j][c].b);
          s[j][c].a = kCut;
        }
        if (j == 0 && ALL)
          m[c] = s[0][c];
        else if (ALL || j < n)
          m[c] = then<RAGGED>(m[c], s[j][c]);
      }
    }
  }
  __device__ __forceinline__ void maps(const Tensors<DT>& t, const Place<V>& at, Map (&m)[V]) {
    if constexpr (RAGGED) cut.find(t.cu, t.n_seqs, s0, n, t.template end<RAGGED>());
#pragma unroll
    for (int c = 0; c < V; ++c) m[c] = {1.0f, 0.0f};
    if (n == LS) maps_of<true>(t, at, m); else maps_of<false>(t, at, m);
  }
  // the states from the one before the steps
  template <bool ALL>
  __device__ __forceinline__ void walk_of(const Tensors<DT>& t, const Place<V>& at, float (&h)[V]) {
    typename C::T* const H = t.H + (at.row * t.T_ + s0) * t.d + at.tile;
#pragma unroll
    for (int j = 0; j < LS; ++j) {
      if (!ALL && j >= n) {
        if (RAGGED && s0 + j < t.T_ && at.live) C{}.store(H + j * t.d, at.off);
        continue;
      }
      C o;
#pragma unroll
      for (int c = 0; c < V; ++c) h[c] = through<RAGGED>(s[j][c], h[c]);
      o.set(h);
      if (at.live) {
        o.store(H + j * t.d, at.off);
        if (t.last && (RAGGED ? (cut.tail >> j) & 1 : s0 + j == t.T_ - 1))
          o.store(t.last + (RAGGED ? cut.seg[j] : at.row) * t.d + at.tile, at.off);
      }
    }
  }
  __device__ __forceinline__ void walk(const Tensors<DT>& t, const Place<V>& at, float (&h)[V]) {
    if (n == LS) walk_of<true>(t, at, h); else walk_of<false>(t, at, h);
  }
  // the state before the row
  static __device__ __forceinline__ void start(const Tensors<DT>& t, const Place<V>& at, float (&h)[V]) {
#pragma unroll
    for (int c = 0; c < V; ++c) h[c] = !RAGGED && t.h0 ? Storage<DT>::load(t.h0 + at.row * t.d + at.tile + at.off + c) : 0.0f;
  }
};

template <int DT, int G, int V, int LS, int NW, bool RAGGED>
__global__ void __launch_bounds__(64 * NW) k_scan_walk(Tensors<DT> t) {
  using W = Fore<DT, G, V, LS, RAGGED>;
  __shared__ Map part[2][NW][V][64];
  const int64_t b = block_in_rows();
  if (b >= t.chains) return;
  const Place<V> at(t.d, b);
  W w[2];
  w[0].load(t, at, 0);
  float h[V];   // the state before the chunk
  W::start(t, at, h);
  auto chunk = [&](W& now, W& next, int64_t k) {
    if (k + 1 < t.chunks) next.load(t, at, (k + 1) * (NW * LS));
    Map m[V];
    now.maps(t, at, m);
    Map(*const p)[V][64] = part[k & 1];
#pragma unroll
    for (int c = 0; c < V; ++c) p[at.wave][c][at.lane] = m[c];
    lds_barrier();
    float mine[V];
#pragma unroll
    for (int v = 0; v < NW; ++v) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        if (v == at.wave) mine[c] = h[c];
        h[c] = through<RAGGED>(p[v][c][at.lane], h[c]);
      }
    }
    now.walk(t, at, mine);
  };
  for (int64_t k = 0; k < t.chunks; k += 2) {
    chunk(w[0], w[1], k);
    if (k + 1 < t.chunks) chunk(w[1], w[0], k + 1);
  }
}

// A ticket's chunk, in the order of the walk, of its chain
__device__ __forceinline__ int64_t take_ticket(unsigned* ticket, unsigned* shared) {
  if (threadIdx.x == 0) *shared = atomicAdd(ticket, 1u);
  __syncthreads();
  return static_cast<unsigned>(__builtin_amdgcn_readfirstlane(*shared));
}

// What the last wave does for all: the waves' maps in `part` (in the order of the
// walk: order(0), order(1), ..) become their carries (the first number of their
// slots), and the chunk's records are published; e: the carry of a chain's first
// chunk.  The state's status goes out by announce after the barrier that follows.
template <int V, int NW, bool CUTS, class Order>
__device__ __forceinline__ void join(const Records& rec, int64_t base, int64_t c, int lane, unsigned spin_limit,
                                     bool map_first, Map (*part)[V][64], float (&e)[V], Order order) {
  Map tot[V];
#pragma unroll
  for (int v = 0; v < V; ++v) tot[v] = part[order(0)][v][lane];
#pragma unroll
  for (int w = 1; w < NW; ++w)
#pragma unroll
    for (int v = 0; v < V; ++v) tot[v] = then<CUTS>(tot[v], part[order(w)][v][lane]);
  if (c > 0) look_back<V, CUTS>(rec, base, c, tot, lane, spin_limit, map_first, e);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    put(rec.states + (base + c) * V * 64 + v * 64 + lane, through<CUTS>(tot[v], e[v]));
    float h = e[v];
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      Map& slot = part[order(w)][v][lane];
      const Map m = slot;
      slot.a = h;
      h = through<CUTS>(m, h);
    }
  }
}

template <int DT, int G, int V, int LS, int NW, bool RAGGED>
__global__ void __launch_bounds__(64 * NW) k_scan_pass(Tensors<DT> t, Records rec, unsigned spin_limit, bool map_first) {
  using W = Fore<DT, G, V, LS, RAGGED>;
  __shared__ Map part[NW][V][64];
  __shared__ unsigned tk;
  const int64_t ticket = take_ticket(rec.ticket, &tk), c = ticket / t.chains;
  if (c >= t.chunks) return;
  const Place<V> at(t.d, ticket - c * t.chains);
  W w;
  w.load(t, at, c * (NW * LS));
  Map m[V];
  w.maps(t, at, m);
#pragma unroll
  for (int v = 0; v < V; ++v) part[at.wave][v][at.lane] = m[v];
  lds_barrier();
  const int64_t base = at.chain * t.chunks;
  if (at.wave == NW - 1) {
    float e[V];
    W::start(t, at, e);
    join<V, NW, RAGGED>(rec, base, c, at.lane, spin_limit, map_first, part, e, [](int k) { return k; });
  }
  lds_barrier();
  if (at.wave == NW - 1) announce(rec.status + base + c, kState, at.lane);
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = part[at.wave][v][at.lane].a;
  w.walk(t, at, h);
}

// ------------------------------------------------------------- backward ----

template <int DT, int G, int V, int LS, bool RAGGED>
struct Back {
  using ST = Storage<DT>;
  using C = Chans<DT, V>;
  C x[LS][G], dh[LS], before;   // before: the state before the chunk
  Gate f[LS][V], i[LS][V];
  float g[LS][V];               // the gradient that arrives at a state from outside
  Cuts<LS> cut;
  int64_t s0;
  int n;

  __device__ __forceinline__ bool head(int j) const { return RAGGED && ((cut.head >> j) & 1); }
  __device__ __forceinline__ bool tail(int j) const { return RAGGED && ((cut.tail >> j) & 1); }
  __device__ __forceinline__ int64_t seg(int j, const Place<V>& at) const { return RAGGED ? static_cast<int64_t>(cut.seg[j]) : at.row; }

  __device__ __forceinline__ void load(const Tensors<DT>& t, const Place<V>& at, int64_t first) {
    s0 = first + at.wave * LS;
    n = static_cast<int>(imax(imin(LS, t.template end<RAGGED>() - s0), 0));
    const int64_t row = at.row * t.T_;
#pragma unroll
    for (int j = 0; j < LS; ++j) {
      const int64_t step = row + imin(s0 + j, t.T_ - 1);   // past the end: the last one, not used
#pragma unroll
      for (int k = 0; k < G; ++k) x[j][k].load(t.x + (step * G + k) * t.d + at.tile, at.off);
      dh[j].load(t.dH + step * t.d + at.tile, at.off);
    }
    if (first > 0) {
      before.load(t.H + (row + first - 1) * t.d + at.tile, at.off);
    } else if (!RAGGED && t.h0) {
      before.load(t.h0 + at.row * t.d + at.tile, at.off);
    } else {
      before = {};
    }
  }
  __device__ __forceinline__ float one(const typename C::T* states, int j, int c, const Tensors<DT>& t, const Place<V>& at) const {
    return ST::load(states + seg(j, at) * t.d + at.tile + at.off + c);
  }
  // the maps of the states over the steps, and of the gradient back over them; ALL: n = LS
  template <bool ALL>
  __device__ __forceinline__ void maps_of(const Tensors<DT>& t, const Place<V>& at, Map (&fore)[V], Map (&back)[V]) {
#pragma unroll
    for (int j = 0; j < LS; ++j) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        f[j][c] = gate_of(x[j][0].at(c));
        i[j][c] = G == 2 ? Gate{f[j][c].off, f[j][c].on} : gate_of(x[j][1].at(c));
        g[j][c] = dh[j].at(c);
        if (!ALL && j >= n) continue;
        if (t.dlast && (RAGGED ? tail(j) : s0 + j == t.T_ - 1)) g[j][c] += one(t.dlast, j, c, t, at);
        Map m = {f[j][c].on, i[j][c].on * x[j][G - 1].at(c)};
        if (head(j)) {
          m.b = fmaf(m.a, t.h0 ? one(t.h0, j, c, t, at) : 0.0f, m.b);
          m.a = kCut;
        }
        fore[c] = ALL && j == 0 ? m : then<RAGGED>(fore[c], m);
      }
    }
#pragma unroll
    for (int j = LS - 1; j >= 0; --j) {
      if (!ALL && j >= n) continue;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const Map m = {tail(j) ? kCut : f[j][c].on, f[j][c].on * g[j][c]};
        back[c] = ALL && j == LS - 1 ? m : then<RAGGED>(back[c], m);
      }
    }
  }
  __device__ __forceinline__ void maps(const Tensors<DT>& t, const Place<V>& at, Map (&fore)[V], Map (&back)[V]) {
    if constexpr (RAGGED) cut.find(t.cu, t.n_seqs, s0, n, t.template end<RAGGED>());
#pragma unroll
    for (int c = 0; c < V; ++c) fore[c] = back[c] = {1.0f, 0.0f};
    if (n == LS) maps_of<true>(t, at, fore, back); else maps_of<false>(t, at, fore, back);
  }
  // the gradients, from the state before the steps and the gradient that arrives at their last state from after it
  template <bool ALL>
  __device__ __forceinline__ void walk_of(const Tensors<DT>& t, const Place<V>& at, float (&h)[V], float (&m)[V]) {
    float prev[LS][V];
#pragma unroll
    for (int j = 0; j < LS; ++j) {
      if (!ALL && j >= n) continue;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        if (head(j)) h[c] = t.h0 ? one(t.h0, j, c, t, at) : 0.0f;
        prev[j][c] = h[c];
        h[c] = fmaf(f[j][c].on, h[c], i[j][c].on * x[j][G - 1].at(c));
      }
    }
    typename ST::T* const dx = t.dx + (at.row * t.T_ + s0) * G * t.d + at.tile;
#pragma unroll
    for (int j = LS - 1; j >= 0; --j) {
      if (!ALL && j >= n) {
#pragma unroll
        for (int k = 0; k < G; ++k)
          if (RAGGED && s0 + j < t.T_ && at.live) C{}.store(dx + (j * G + k) * t.d, at.off);
        continue;
      }
      float o[G][V];
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float lam = tail(j) ? g[j][c] : g[j][c] + m[c], val = x[j][G - 1].at(c);
        o[0][c] = lam * (G == 2 ? prev[j][c] - val : prev[j][c]) * (f[j][c].on * f[j][c].off);
        if constexpr (G == 3) o[1][c] = lam * val * (i[j][c].on * i[j][c].off);
        o[G - 1][c] = lam * i[j][c].on;
        m[c] = f[j][c].on * lam;
      }
      if (at.live) {
        C out;
#pragma unroll
        for (int k = 0; k < G; ++k) {
          out.set(o[k]);
          out.store(dx + (j * G + k) * t.d, at.off);
        }
        if (t.dh0 && (RAGGED ? head(j) : s0 + j == 0)) {
          out.set(m);
          out.store(t.dh0 + seg(j, at) * t.d + at.tile, at.off);
        }
      }
    }
  }
  __device__ __forceinline__ void walk(const Tensors<DT>& t, const Place<V>& at, float (&h)[V], float (&m)[V]) {
    if (n == LS) walk_of<true>(t, at, h, m); else walk_of<false>(t, at, h, m);
  }
  // the state before this wave's steps, through the waves' maps before it
  template <int NW>
  __device__ __forceinline__ void entry(const Place<V>& at, const Map (*fore)[V][64], float (&h)[V]) const {
#pragma unroll
    for (int c = 0; c < V; ++c) h[c] = before.at(c);
#pragma unroll
    for (int w = 0; w < NW - 1; ++w) {
      if (w >= at.wave) break;
#pragma unroll
      for (int c = 0; c < V; ++c) h[c] = through<RAGGED>(fore[w][c][at.lane], h[c]);
    }
  }
};

template <int DT, int G, int V, int LS, int NW, bool RAGGED>
__global__ void __launch_bounds__(64 * NW) k_scan_walk_back(Tensors<DT> t) {
  using W = Back<DT, G, V, LS, RAGGED>;
  __shared__ Map fore[2][NW][V][64], back[2][NW][V][64];
  const int64_t b = block_in_rows();
  if (b >= t.chains) return;
  const Place<V> at(t.d, b);
  auto first = [&](int64_t k) { return (t.chunks - 1 - k) * (NW * LS); };   // chunk k from the end
  W w[2];
  w[0].load(t, at, first(0));
  float mu[V];   // the gradient that arrives at the chunk's last state from the steps after it
#pragma unroll
  for (int c = 0; c < V; ++c) mu[c] = 0.0f;
  auto chunk = [&](W& now, W& next, int64_t k) {
    if (k + 1 < t.chunks) next.load(t, at, first(k + 1));
    Map mf[V], mb[V];
    now.maps(t, at, mf, mb);
    Map(*const pf)[V][64] = fore[k & 1], (*const pb)[V][64] = back[k & 1];
#pragma unroll
    for (int c = 0; c < V; ++c) {
      pf[at.wave][c][at.lane] = mf[c];
      pb[at.wave][c][at.lane] = mb[c];
    }
    lds_barrier();
    float h[V], m[V];
    now.template entry<NW>(at, pf, h);
#pragma unroll
    for (int v = NW - 1; v >= 0; --v) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        if (v == at.wave) m[c] = mu[c];
        mu[c] = through<RAGGED>(pb[v][c][at.lane], mu[c]);
      }
    }
    now.walk(t, at, h, m);
  };
  for (int64_t k = 0; k < t.chunks; k += 2) {
    chunk(w[0], w[1], k);
    if (k + 1 < t.chunks) chunk(w[1], w[0], k + 1);
  }
}

template <int DT, int G, int V, int LS, int NW, bool RAGGED>
__global__ void __launch_bounds__(64 * NW) k_scan_pass_back(Tensors<DT> t, Records rec, unsigned spin_limit, bool map_first) {
  using W = Back<DT, G, V, LS, RAGGED>;
  __shared__ Map fore[NW][V][64], back[NW][V][64];
  __shared__ unsigned tk;
  const int64_t ticket = take_ticket(rec.ticket, &tk), c = ticket / t.chains;   // c: from the end
  if (c >= t.chunks) return;
  const Place<V> at(t.d, ticket - c * t.chains);
  W w;
  w.load(t, at, (t.chunks - 1 - c) * (NW * LS));
  Map mf[V], mb[V];
  w.maps(t, at, mf, mb);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    fore[at.wave][v][at.lane] = mf[v];
    back[at.wave][v][at.lane] = mb[v];
  }
  lds_barrier();
  const int64_t base = at.chain * t.chunks;
  if (at.wave == NW - 1) {
    float e[V] = {};
    join<V, NW, RAGGED>(rec, base, c, at.lane, spin_limit, map_first, back, e, [](int k) { return NW - 1 - k; });
  }
  lds_barrier();
  if (at.wave == NW - 1) announce(rec.status + base + c, kState, at.lane);
  float h[V], m[V];
  w.template entry<NW>(at, fore, h);
#pragma unroll
  for (int v = 0; v < V; ++v) m[v] = back[at.wave][v][at.lane].a;
  w.walk(t, at, h, m);
}

// What comes before: the words that a call's records begin with become zero, and
// out[j] = in[j] (0 without in) for the sequences of a pack that have no step, or,
// without cu, for every row.
template <class T>
__global__ void __launch_bounds__(256) k_scan_begin(unsigned* __restrict__ words, int64_t n, const int32_t* __restrict__ cu,
                                                    int64_t rows, int64_t d, const T* __restrict__ in, T* __restrict__ out) {
  int64_t i = block_in_rows() * 256 + threadIdx.x;
  if (i < n) {
    words[i] = 0;
    return;
  }
  i -= n;
  if (i >= rows * d) return;
  const int64_t j = i / d;
  if (cu && cu[j + 1] > cu[j]) return;
  out[i] = in ? in[i] : T(0);
}

// ---------------------------------------------------------------- plan ----

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up(size_t x) { return (x + 255) / 256 * 256; }

// Chains from which a workgroup each fills the device, and steps up to which a
// few chunks one after another take no longer than the look-back and the launch
// that clears its records.  (Taking the maps of 512 stretches of time first, by a
// kernel of their own that reads the inputs once more, took 43 and 65 us for 8 x
// 4096 x 512 bf16, 284 and 400 for 2 x 131072 x 256 fp32, where look-back takes 29
// and 46, 174 and 272.  Tiles of 16 channels, so that every one of 8 x 512 has a
// chain that fills the device: 40 and 73.)
constexpr int64_t kEnough = 256, kShort = 256, kCus = 256;
// Steps of a wave and waves of a workgroup.  A longer chunk means fewer
// look-backs in a row, as long as the registers allow a workgroup of it, or two
// of the smaller ones, on a CU.  us, glr, 2 x 131072 x 256 fp32 and 8 x 4096 x 512
// bf16, steps x waves: forward 16 x 16 174 and 29, 12 x 16 187 and 32, 16 x 12 178 and
// 32 (8 x 16 and 8 waves were 10 to 50% slower); backward 16 x 8 272, 8 x 16 46 (8 x 8
// and 12 x 8 5 to 25% slower, 4 x 16 half as long again).  Where a workgroup has
// its chain (64 x 1024 x 512 bf16), 8 x 8 took as long as 8 x 16 and 8 x 12 or less,
// 4 x 8, 4 x 16 and 16 x 8 10 to 25% longer.
struct Shape {
  int steps, waves;
  constexpr int chunk() const { return steps * waves; }
};
template <int G, int V>
constexpr Shape shape_of(bool back, bool pass) {
  if (!pass) return {8, 8};
  if (!back) return {16, 16};
  if (V == 1) return G == 2 ? Shape{16, 8} : Shape{8, 16};
  return G == 2 ? Shape{8, 16} : Shape{8, 8};   // (glri of two channels a lane: more than 128 registers)
}
// A longer one for rows of one channel a lane, of as many waves: such a workgroup
// has a CU to itself, so it is taken where it makes fewer steps of rounds of the
// device.  us, 20011 x 250 fp32 glri in 37 sequences (four chains): forward 20 steps, one round,
// 26, 16 steps, two, 35; backward 10 steps, two rounds, 43, 8 steps, three, 48.
// (24 steps 35; 12 steps backward 57.)  The two lengths are of this shape alone.
template <int G, int V>
constexpr Shape longer_of(bool back) {
  const Shape s = shape_of<G, V>(back, true);
  if (V > 1) return s;
  return back ? G == 3 ? Shape{10, s.waves} : s : Shape{20, s.waves};
}
Shape longer_of(int G, int V, bool back) {
  if (V > 1) return G == 2 ? longer_of<2, 2>(back) : longer_of<3, 2>(back);
  return G == 2 ? longer_of<2, 1>(back) : longer_of<3, 1>(back);
}
Shape shape_of(int G, int V, bool back, bool pass) {
  if (G == 2) return V == 1 ? shape_of<2, 1>(back, pass) : shape_of<2, 2>(back, pass);
  return V == 1 ? shape_of<3, 1>(back, pass) : shape_of<3, 2>(back, pass);
}

struct Plan {
  int V;
  bool pass, longer;
  int64_t chains, chunks;
  size_t words, maps_off, states_off, total;
};
Plan plan_of(const GatedScanArgs& a, bool back) {
  Plan p{};
  if (a.T == 0) return p;
  p.V = a.bf16 && a.d % 2 == 0 ? 2 : 1;   // 4 bytes a lane where the rows allow it
  p.chains = a.B * cdiv(a.d, 64 * p.V);
  p.pass = p.chains < kEnough && a.T > kShort;
  Shape s = shape_of(a.G, p.V, back, p.pass);
  if (p.pass) {
    const Shape l = longer_of(a.G, p.V, back);
    auto steps = [&](const Shape& k) { return cdiv(p.chains * cdiv(a.T, k.chunk()), kCus) * k.steps; };
    p.longer = steps(l) < steps(s);
    if (p.longer) s = l;
  }
  p.chunks = cdiv(a.T, s.chunk());
  if (p.pass) {
    const size_t n = size_t(p.chains) * p.chunks, line = size_t(p.V) * 64 * sizeof(float);
    p.words = 2 + n;   // ticket, error, statuses
    p.maps_off = up(p.words * sizeof(unsigned));
    p.states_off = p.maps_off + up(n * 2 * line);
    p.total = p.states_off + up(n * line);
  }
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

// the records of a call that has some, and `out` of the sequences without a step
Records begin(const GatedScanArgs& a, const Plan& p, const void* in, void* out) {
  unsigned* const words = reinterpret_cast<unsigned*>(a.ws);
  const int64_t rows = !out || (a.n_seqs == 0 && a.T > 0) ? 0 : a.n_seqs > 0 ? a.n_seqs : a.B;
  const int64_t n = static_cast<int64_t>(p.words) + rows * a.d;
  const dim3 grid = rows_of_blocks(cdiv(n, 256));
  if (n > 0 && a.bf16)
    k_scan_begin<uint16_t><<<grid, 256, 0, a.stream>>>(words, p.words, a.cu, rows, a.d, static_cast<const uint16_t*>(in),
                                                       static_cast<uint16_t*>(out));
  else if (n > 0)
    k_scan_begin<float><<<grid, 256, 0, a.stream>>>(words, p.words, a.cu, rows, a.d, static_cast<const float*>(in),
                                                    static_cast<float*>(out));
  return {words, a.error ? a.error : words + 1, words + 2, reinterpret_cast<float*>(a.ws + p.maps_off),
          reinterpret_cast<float*>(a.ws + p.states_off)};
}

template <int DT>
Tensors<DT> tensors_of(const GatedScanArgs& a, const Plan& p) {
  using T = typename Storage<DT>::T;
  return {static_cast<const T*>(a.xproj), static_cast<const T*>(a.h0), static_cast<const T*>(a.dH), static_cast<const T*>(a.dlast),
          static_cast<T*>(a.H), static_cast<T*>(a.last), static_cast<T*>(a.dxproj), static_cast<T*>(a.dh0),
          a.cu, a.n_seqs, a.B, a.T, a.d, p.chains, p.chunks};
}

}  // namespace

bool gated_scan_fits(const GatedScanArgs& a) {
  // a ticket counts the chunks of all chains; a chunk has 64 steps or more
  return double(a.B) * (double(a.d) / 64 + 1) * (double(a.T) / 64 + 1) < 4194304.0 * 512;
}
size_t gated_scan_workspace(const GatedScanArgs& a) { return plan_of(a, false).total; }
size_t gated_scan_backward_workspace(const GatedScanArgs& a) { return plan_of(a, true).total; }

void launch_gated_scan(const GatedScanArgs& a) {
  const Plan p = plan_of(a, false);
  const Records rec = begin(a, p, a.h0, a.last);
  if (a.T == 0) return;
  typed(a, p.V, [&](auto dt, auto g, auto v, auto ragged) {
    constexpr int DT = decltype(dt)::value, G = decltype(g)::value, V = decltype(v)::value;
    constexpr bool RAGGED = decltype(ragged)::value;
    const Tensors<DT> t = tensors_of<DT>(a, p);
    constexpr Shape pass = shape_of<G, V>(false, true), longer = longer_of<G, V>(false), walk = shape_of<G, V>(false, false);
    if (longer.steps > pass.steps && p.longer)
      k_scan_pass<DT, G, V, longer.steps, longer.waves, RAGGED>
          <<<rows_of_blocks(p.chains * p.chunks), 64 * longer.waves, 0, a.stream>>>(t, rec, a.spin_limit, p.chains < 64);
    else if (p.pass)
      k_scan_pass<DT, G, V, pass.steps, pass.waves, RAGGED><<<rows_of_blocks(p.chains * p.chunks), 64 * pass.waves, 0, a.stream>>>(
          t, rec, a.spin_limit, p.chains < 64);
    else
      k_scan_walk<DT, G, V, walk.steps, walk.waves, RAGGED><<<rows_of_blocks(p.chains), 64 * walk.waves, 0, a.stream>>>(t);
  });
}

void launch_gated_scan_backward(const GatedScanArgs& a) {
  const Plan p = plan_of(a, true);
  const Records rec = begin(a, p, a.dlast, a.dh0);
  if (a.T == 0) return;
  typed(a, p.V, [&](auto dt, auto g, auto v, auto ragged) {
    constexpr int DT = decltype(dt)::value, G = decltype(g)::value, V = decltype(v)::value;
    constexpr bool RAGGED = decltype(ragged)::value;
    const Tensors<DT> t = tensors_of<DT>(a, p);
    constexpr Shape pass = shape_of<G, V>(true, true), longer = longer_of<G, V>(true), walk = shape_of<G, V>(true, false);
    if (longer.steps > pass.steps && p.longer)
      k_scan_pass_back<DT, G, V, longer.steps, longer.waves, RAGGED>
          <<<rows_of_blocks(p.chains * p.chunks), 64 * longer.waves, 0, a.stream>>>(t, rec, a.spin_limit, p.chains < 64);
    else if (p.pass)
      k_scan_pass_back<DT, G, V, pass.steps, pass.waves, RAGGED><<<rows_of_blocks(p.chains * p.chunks), 64 * pass.waves, 0, a.stream>>>(
          t, rec, a.spin_limit, p.chains < 64);
    else
      k_scan_walk_back<DT, G, V, walk.steps, walk.waves, RAGGED><<<rows_of_blocks(p.chains), 64 * walk.waves, 0, a.stream>>>(t);
  });
}

}  // namespace prn
