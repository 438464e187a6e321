// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[n] = s table[tok n]           dtable[v] = s sum over n with tok n = v of dout[n]
//
// Both are bound by memory: the lookup reads a row and writes a row per
// token; the gradient reads every row of dout once and writes every row of
// dtable.  The gradient sums without atomics: the token positions are sorted
// by token (a stable radix sort, so that equal tokens keep their order), and
// every token's rows are then added in that order in fp32.  A token that
// occurs kLong times or more is cut into chunks of kLong rows, whose sums are
// added in order by a second kernel, so that one frequent token does not hold
// up the device.  Rows of no token are cleared beside the sort.
#include "embed.h"

#include <algorithm>
#include <type_traits>

#include "grid_rows.h"
#include "prn_device.h"

namespace prn {
namespace {

constexpr int64_t kNoPad = INT64_MIN;
constexpr int kSortThr = 512;
constexpr int kMaxBits = 9;     // of a radix pass
constexpr int kBins = 1 << kMaxBits;
constexpr int kBlock = 16;      // sorted positions a group of lanes starts from
constexpr int kLong = 16;       // rows of a chunk of a frequent token (a multiple of kBlock)

// VEC elements (16 bytes, or one element where a row is shorter than that) at
// any element's address: global memory takes unaligned vector accesses, so
// odd widths need no narrower path.  A row's last vector is moved back to end
// with the row; the channels two lanes then share get the same value from both.
template <int DT, int VEC>
struct __attribute__((packed, aligned(sizeof(typename Storage<DT>::T)))) Vec {
  typename Storage<DT>::T v[VEC];
};
template <int DT> constexpr int kVec = 16 / sizeof(typename Storage<DT>::T);

template <int DT, int VEC>
__device__ __forceinline__ void unpack(const Vec<DT, VEC>& q, float* o) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) o[e] = Storage<DT>::load(&q.v[e]);
}
template <int DT, int VEC>
__device__ __forceinline__ Vec<DT, VEC> load_vec(const typename Storage<DT>::T* p) {
  return *reinterpret_cast<const Vec<DT, VEC>*>(p);
}
template <int DT, int VEC>
__device__ __forceinline__ void store_vec(typename Storage<DT>::T* p, const float* o) {
  Vec<DT, VEC> q;
#pragma unroll
  for (int e = 0; e < VEC; ++e) q.v[e] = Storage<DT>::pack(o[e]);
  *reinterpret_cast<Vec<DT, VEC>*>(p) = q;
}

__device__ __forceinline__ int64_t token_at(const void* tokens, int bytes, int64_t n) {
  return bytes == 4 ? static_cast<int64_t>(static_cast<const int32_t*>(tokens)[n])
                    : static_cast<const int64_t*>(tokens)[n];
}

// TPR lanes per row, kRows rows of a group in flight.  The pad token's rows
// are zeros, a token outside the table gives NaN.
constexpr int kRows = 4;
template <int DT, int VEC, int TPR>
__global__ void __launch_bounds__(256) k_embed(const void* __restrict__ tokens, int token_bytes,
                                               const typename Storage<DT>::T* __restrict__ table, int64_t N, int64_t V,
                                               int64_t d, float scale, int64_t pad,
                                               typename Storage<DT>::T* __restrict__ out) {
  const int64_t n0 = (block_in_rows() * (256 / TPR) + threadIdx.x / TPR) * kRows;
  int64_t tok[kRows];
#pragma unroll
  for (int q = 0; q < kRows; ++q) tok[q] = n0 + q < N ? token_at(tokens, token_bytes, n0 + q) : -1;
  for (int64_t c = static_cast<int64_t>(threadIdx.x % TPR) * VEC; c < d; c += TPR * VEC) {
    const int64_t cc = imin(c, d - VEC);
    Vec<DT, VEC> raw[kRows];
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      const bool in = tok[q] >= 0 && tok[q] < V && tok[q] != pad;
      raw[q] = load_vec<DT, VEC>(table + (in ? tok[q] : 0) * d + cc);
    }
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      const bool in = tok[q] >= 0 && tok[q] < V && tok[q] != pad;
      const float fill = tok[q] == pad && pad != kNoPad ? 0.0f : __builtin_nanf("");
      float v[VEC];
      unpack<DT, VEC>(raw[q], v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = in ? v[e] * scale : fill;
      if (n0 + q < N) store_vec<DT, VEC>(out + (n0 + q) * d + cc, v);
    }
  }
}

// ----------------------------------------------------------------- sort ---

// a token's sort key: itself, or V where it has no gradient
__device__ __forceinline__ uint32_t key_of(int64_t t, int64_t V, int64_t pad) {
  return t >= 0 && t < V && t != pad ? static_cast<uint32_t>(t) : static_cast<uint32_t>(V);
}

struct SortIn {
  const void* tokens;   // the first pass reads the tokens themselves
  int token_bytes;
  int64_t V, pad;
  const uint32_t *keys, *pos;
};
template <bool FIRST>
__device__ __forceinline__ uint32_t sort_key(const SortIn& in, int64_t i) {
  if constexpr (FIRST) return key_of(token_at(in.tokens, in.token_bytes, i), in.V, in.pad);
  return in.keys[i];
}

// Workgroups below n_tiles: the tile's count of every digit.  The others
// clear their part of dtable (words of 16 bytes).
template <bool FIRST, int ITEMS>
__global__ void __launch_bounds__(kSortThr) k_embed_count(SortIn in, int64_t N, int shift, int bits, int n_tiles,
                                                          uint32_t* __restrict__ counts, uint4* __restrict__ clear,
                                                          int64_t n_clear, uint8_t* __restrict__ tail, int n_tail) {
  if (static_cast<int>(blockIdx.x) >= n_tiles) {
    const int64_t me = (static_cast<int64_t>(blockIdx.x) - n_tiles) * kSortThr + threadIdx.x;
    const int64_t all = (static_cast<int64_t>(gridDim.x) - n_tiles) * kSortThr;
    for (int64_t i = me; i < n_clear; i += all) clear[i] = make_uint4(0, 0, 0, 0);
    if (me < n_tail) tail[me] = 0;
    return;
  }
  __shared__ uint32_t hist[kBins];
  for (int b = threadIdx.x; b < kBins; b += kSortThr) hist[b] = 0;
  __syncthreads();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * (ITEMS * kSortThr);
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const int64_t i = at + j * kSortThr + threadIdx.x;
    if (i < N) atomicAdd(&hist[(sort_key<FIRST>(in, i) >> shift) & ((1u << bits) - 1)], 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < (1 << bits); b += kSortThr)
    counts[static_cast<int64_t>(blockIdx.x) * kBins + b] = hist[b];
}

// Where there are many tiles, the scatter below does not add up the counts of
// all of them, which is quadratic: these are made exclusive sums before it.  A
// workgroup takes `per` rows of counts (a digit a thread), in place, their sums
// to row blockIdx.x of sums; once over the tiles in groups of kGroup, and once
// over the groups, which leaves the digits' totals in sums' last row.
constexpr int kGroup = 256;
__global__ void __launch_bounds__(kSortThr) k_embed_offsets(uint32_t* __restrict__ counts, int n, int per,
                                                            uint32_t* __restrict__ sums) {
  const int tid = threadIdx.x, t0 = static_cast<int>(blockIdx.x) * per, t1 = min(t0 + per, n);
  constexpr int kAhead = 32;
  uint32_t run = 0;
  for (int t = t0; t < t1; t += kAhead) {
    uint32_t c[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) c[q] = t + q < t1 ? counts[static_cast<int64_t>(t + q) * kBins + tid] : 0;
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      if (t + q < t1) counts[static_cast<int64_t>(t + q) * kBins + tid] = run;
      run += c[q];
    }
  }
  sums[static_cast<int64_t>(blockIdx.x) * kBins + tid] = run;
}

// The lanes of the wave that hold the same digit (of `bits` bits), this one
// among them; live lanes only.
__device__ __forceinline__ unsigned long long same_digit(uint32_t dg, int bits, bool live) {
  unsigned long long same = __ballot(live);
#pragma unroll
  for (int b = 0; b < kMaxBits; ++b) {
    if (b < bits) {
      const bool on = (dg >> b) & 1;
      const unsigned long long m = __ballot(on);
      same &= on ? m : ~m;
    }
  }
  return same;
}
// inclusive sum over the wave
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = __shfl_up(v, o, 64);
    if (lane >= o) v += up;
  }
  return v;
}

// Stable scatter by one digit.  A wave of a tile holds 64 ITEMS positions in
// order; a position's rank among the equal digits before it in the wave comes
// from ballots, the counts of earlier waves, tiles and digits are added to it
// (groups > 0: those of tiles and digits as k_embed_offsets leaves them).
template <bool FIRST, int ITEMS>
__global__ void __launch_bounds__(kSortThr) k_embed_scatter(SortIn in, int64_t N, int shift, int bits, int n_tiles,
                                                            const uint32_t* __restrict__ counts,
                                                            const uint32_t* __restrict__ sums, int groups,
                                                            uint32_t* __restrict__ keys_out,
                                                            uint32_t* __restrict__ pos_out) {
  constexpr int NW = kSortThr / 64;
  static_assert(kBins == kSortThr, "a digit a thread");
  __shared__ uint32_t wave_hist[NW][kBins];
  __shared__ uint32_t scan[NW];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int nb = 1 << bits, me = static_cast<int>(blockIdx.x);
  const int64_t at = (static_cast<int64_t>(me) * NW + w) * (64 * ITEMS);
  uint32_t key[ITEMS], pos[ITEMS], rank[ITEMS];
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const int64_t i = at + j * 64 + lane;
    key[j] = i < N ? sort_key<FIRST>(in, i) : 0;
    pos[j] = FIRST ? static_cast<uint32_t>(i) : i < N ? in.pos[i] : 0;
  }
  // this thread's digit: its count in all tiles, and in the tiles before this one
  uint32_t total = 0, before = 0;
  if (groups > 0) {
    if (tid < nb) {
      total = sums[static_cast<int64_t>(groups) * kBins + tid];
      before = sums[static_cast<int64_t>(me / kGroup) * kBins + tid] + counts[static_cast<int64_t>(me) * kBins + tid];
    }
  } else if (tid < nb) {
    int t = 0;
    for (; t + 32 <= n_tiles; t += 32) {
      uint32_t c[32];
#pragma unroll
      for (int q = 0; q < 32; ++q) c[q] = counts[static_cast<int64_t>(t + q) * kBins + tid];
#pragma unroll
      for (int q = 0; q < 32; ++q) {
        total += c[q];
        before += t + q < me ? c[q] : 0;
      }
    }
#pragma unroll 8
    for (; t < n_tiles; ++t) {
      const uint32_t c = counts[static_cast<int64_t>(t) * kBins + tid];
      total += c;
      before += t < me ? c : 0;
    }
  }
  for (int b = lane; b < nb; b += 64) wave_hist[w][b] = 0;
  // other lanes of the wave write it between two reads; a wave's LDS accesses are done in order
  volatile uint32_t* const mine_hist = wave_hist[w];
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const bool live = at + j * 64 + lane < N;
    const uint32_t dg = (key[j] >> shift) & (nb - 1);
    const unsigned long long same = same_digit(dg, bits, live);
    if (live) {
      const uint32_t sofar = mine_hist[dg];
      rank[j] = sofar + __popcll(same & ((1ull << lane) - 1));
      if ((same >> lane) == 1ull) mine_hist[dg] = sofar + __popcll(same);   // the last lane of the digit counts them all
    }
  }
  // exclusive sum of the totals over the digits
  const uint32_t incl = wave_scan(total);
  if (lane == 63) scan[w] = incl;
  __syncthreads();   // also: every wave's histogram is complete
  uint32_t base = incl - total + before;
  for (int q = 0; q < w; ++q) base += scan[q];
  if (tid < nb) {    // where each wave's first position of the digit goes
#pragma unroll
    for (int q = 0; q < NW; ++q) {
      const uint32_t c = wave_hist[q][tid];
      wave_hist[q][tid] = base;
      base += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    if (at + j * 64 + lane < N) {
      const uint32_t to = wave_hist[w][(key[j] >> shift) & (nb - 1)] + rank[j];
      keys_out[to] = key[j];
      pos_out[to] = pos[j];
    }
  }
}

// ----------------------------------------------------------------- sums ---

// the first i in [0, n) with keys[i] >= k (n if none); the whole wave searches
__device__ __forceinline__ int64_t lower_bound(const uint32_t* keys, int64_t n, uint32_t k) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t step = (hi - lo + 63) / 64, i = lo + lane * step;
    const int less = __popcll(__ballot(i < hi && keys[i < hi ? i : lo] < k));   // a leading run of lanes
    if (less == 0) return lo;
    hi = imin(hi, lo + less * step);
    lo += (less - 1) * step + 1;
  }
  return lo;
}

// Sums the rows i0 .. i1 - 1 at channels c .., in order, into acc: where(i) is
// row i's position in dout (wave-uniform); emit(i, acc) is called before row i
// is added and may hand acc on and restart it.
constexpr int kBatch = 8;   // rows in flight
template <int DT, int VEC, class Where, class Emit>
__device__ __forceinline__ void walk_rows(const typename Storage<DT>::T* dout, int64_t d, int64_t c, bool mine, int i0,
                                          int i1, Where where, Emit emit, float* acc) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.0f;
  for (int i = i0; i < i1; i += kBatch) {
    Vec<DT, VEC> raw[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      if (i + q < i1 && mine) raw[q] = load_vec<DT, VEC>(dout + static_cast<int64_t>(where(i + q)) * d + c);
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      if (i + q < i1) {
        emit(i + q, acc);
        float v[VEC];
        unpack<DT, VEC>(raw[q], v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += v[e];
      }
    }
  }
}

// A wave per kBlock sorted positions and 64 VEC channels (blockIdx.z): sums
// every token whose rows start there, and the chunk of a frequent token from
// an earlier block that starts there (at most one: chunks are kLong >= kBlock
// apart).  A frequent token's chunks go to part: its first to row 2 block + 1,
// the others to row 2 block.  The keys and positions of the 64 sorted places a
// wave may need (kBlock - 1 + kLong of them) are loaded at once; every decision
// after that is a ballot.
template <int DT, int VEC>
__global__ void __launch_bounds__(256) k_embed_sum(const uint32_t* __restrict__ keys, const uint32_t* __restrict__ pos,
                                                   const typename Storage<DT>::T* __restrict__ dout, int64_t N, int64_t V,
                                                   int64_t d, float scale, typename Storage<DT>::T* __restrict__ dtable,
                                                   float* __restrict__ part) {
  constexpr uint32_t kNone = 0xffffffffu;   // above every key
  const int lane = threadIdx.x & 63;
  const int64_t block = block_in_rows() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t p0 = block * kBlock;
  if (p0 >= N) return;
  const int64_t c0 = (static_cast<int64_t>(blockIdx.z) * 64 + lane) * VEC, c = imin(c0, d - VEC);
  const bool mine = c0 < d;
  // lane t + 1: place t (position p0 + t), the place before p0 in lane 0
  static_assert(kBlock + kLong <= 63, "the places fit a wave");
  const int64_t ia = p0 - 1 + lane;
  const uint32_t ka = ia >= 0 && ia < N ? keys[ia] : kNone, qa = ia >= 0 && ia < N ? pos[ia] : 0;
  const uint32_t prev = __shfl_up(ka, 1, 64), later = __shfl_down(ka, kLong - 1, 64);
  // bit t: place t holds another key than place t - 1
  const unsigned long long turn = __ballot(lane >= 1 && ka != prev) >> 1;
  const unsigned own = static_cast<unsigned>(turn & __ballot(ka < V) >> 1) & ((1u << kBlock) - 1);
  const unsigned frequent = own & static_cast<unsigned>(__ballot(ka == later) >> 1);
  float acc[VEC];
  auto to_part = [&](int64_t row) {
    if (mine) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) part[row * d + c + e] = acc[e];
    }
  };

  const uint32_t k0 = __shfl(ka, 1, 64);
  if (!(turn & 1) && k0 < V) {
    // a token from an earlier block: its chunk that starts here, if it is a frequent one
    const int64_t s = lower_bound(keys, p0, k0);
    if (s + kLong <= N && keys[s + kLong - 1] == k0) {
      const int64_t b = s + (p0 - s + kLong - 1) / kLong * kLong;
      const bool in = lane < kLong && b + lane < N;
      const unsigned long long run = __ballot(in && keys[in ? b + lane : 0] == k0);
      const uint32_t at = in ? pos[b + lane] : 0;
      if (b < p0 + kBlock && (run & 1)) {
        const int n = __builtin_ctzll(~run);   // up to kLong
        walk_rows<DT, VEC>(dout, d, c, mine, 0, n, [&](int i) { return __builtin_amdgcn_readlane(at, i); },
                           [](int, float*) {}, acc);
        to_part(2 * block);
      }
    }
  }
  if (!own) return;
  const int t0 = __builtin_ctz(own), t1 = 31 - __builtin_clz(own);   // first and last token that starts here
  const bool last_frequent = (frequent >> t1) & 1;
  // a shorter run ends within kLong places
  const int end = last_frequent ? t1 + kLong : t1 + 1 + __builtin_ctzll(turn >> (t1 + 1));
  uint32_t token = __builtin_amdgcn_readlane(ka, t0 + 1);
  auto to_table = [&]() {
    if (mine) {
      float o[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) o[e] = acc[e] * scale;
      store_vec<DT, VEC>(dtable + static_cast<int64_t>(token) * d + c, o);
    }
  };
  walk_rows<DT, VEC>(
      dout, d, c, mine, t0, end,
      [&](int t) { return __builtin_amdgcn_readlane(qa, t + 1); },
      [&](int t, float* s) {
        if (t > t0 && t <= t1 && ((own >> t) & 1)) {
          to_table();
          token = __builtin_amdgcn_readlane(ka, t + 1);
#pragma unroll
          for (int e = 0; e < VEC; ++e) s[e] = 0.0f;
        }
      },
      acc);
  if (last_frequent)
    to_part(2 * block + 1);
  else
    to_table();
}

// The frequent tokens that start among kJoin sorted positions: their chunks'
// sums at 64 CPT channels (blockIdx.z), added in order, a wave per token; a
// token of kMany chunks or more by all 16 waves (every 16th chunk each, then
// the waves in order).  All waves for every token took 37 us at 262144 tokens
// over 131072, where up to 16 tokens start in one workgroup; this takes 30, most
// of it the 22000 rows of the most frequent token in one workgroup.
constexpr int kJoin = 256, kJoinThr = 1024, kJoinBatch = 8, kMany = 33;
template <int DT, int CPT>
__global__ void __launch_bounds__(kJoinThr) k_embed_join(const uint32_t* __restrict__ keys, const float* __restrict__ part,
                                                         int64_t N, int64_t V, int64_t d, float scale,
                                                         typename Storage<DT>::T* __restrict__ dtable) {
  using F = Vec<kF32, CPT>;
  constexpr int NW = kJoinThr / 64;
  static_assert(kMany <= 64, "a wave counts its chunks at once");
  __shared__ uint32_t n_found, n_many;
  __shared__ uint32_t found[kJoin / kLong + 1], many[kJoin / kLong + 1];
  __shared__ float hand[NW][64 * CPT];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t at = block_in_rows() * kJoin;
  const int64_t p = at + threadIdx.x;
  bool starts = false;
  if (threadIdx.x < kJoin && p + kLong <= N) {
    const uint32_t k = keys[p];
    starts = k < V && keys[p + kLong - 1] == k && (p == 0 || keys[p - 1] != k);
  }
  if (threadIdx.x == 0) n_found = n_many = 0;
  __syncthreads();
  if (starts) found[atomicAdd(&n_found, 1u)] = threadIdx.x;
  __syncthreads();
  const int64_t c0 = (static_cast<int64_t>(blockIdx.z) * 64 + lane) * CPT, c = imin(c0, d - CPT);
  const bool mine = c0 < d;
  // how many of the token's chunks from q0 on there are, up to 64: chunk q is
  // there if its first position holds the token
  auto chunks = [&](int64_t s, uint32_t k, int64_t q0) {
    const int64_t i = s + (q0 + lane) * kLong;
    const unsigned long long there = __ballot(i < N && keys[i < N ? i : s] == k);
    return ~there == 0 ? 64 : __builtin_ctzll(~there);
  };
  // acc += the sums of chunks q0 + first, + every .. of q0 + n
  auto add = [&](int64_t s, int64_t q0, int first, int every, int n, float* acc) {
    if (!mine) return;
    for (int q = first; q < n; q += every * kJoinBatch) {
      F v[kJoinBatch];
#pragma unroll
      for (int b = 0; b < kJoinBatch; ++b) {
        const int64_t qq = q0 + q + b * every;
        if (q + b * every < n) v[b] = *reinterpret_cast<const F*>(part + (2 * ((s + qq * kLong) / kBlock) + (qq == 0)) * d + c);
      }
#pragma unroll
      for (int b = 0; b < kJoinBatch; ++b)
        if (q + b * every < n) {
#pragma unroll
          for (int e = 0; e < CPT; ++e) acc[e] += v[b].v[e];
        }
    }
  };
  auto finish = [&](uint32_t k, float* acc) {
    if (!mine) return;
#pragma unroll
    for (int e = 0; e < CPT; ++e) acc[e] *= scale;
    store_vec<DT, CPT>(dtable + static_cast<int64_t>(k) * d + c, acc);
  };
  for (uint32_t f = w; f < n_found; f += NW) {   // in any order: each writes its own row
    const int64_t s = at + __builtin_amdgcn_readfirstlane(found[f]);
    const uint32_t k = __builtin_amdgcn_readfirstlane(keys[s]);
    const int n = chunks(s, k, 0);
    if (n >= kMany) {
      if (lane == 0) many[atomicAdd(&n_many, 1u)] = found[f];
      continue;
    }
    float acc[CPT] = {};
    add(s, 0, 0, 1, n, acc);
    finish(k, acc);
  }
  __syncthreads();
  for (uint32_t f = 0; f < n_many; ++f) {
    const int64_t s = at + __builtin_amdgcn_readfirstlane(many[f]);
    const uint32_t k = __builtin_amdgcn_readfirstlane(keys[s]);
    float acc[CPT] = {};
    for (int64_t q0 = 0;; q0 += 64) {
      const int n = chunks(s, k, q0);
      add(s, q0, w, NW, n, acc);
      if (n < 64) break;
    }
#pragma unroll
    for (int e = 0; e < CPT; ++e) hand[w][lane * CPT + e] = acc[e];
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int q = 1; q < NW; ++q)
#pragma unroll
        for (int e = 0; e < CPT; ++e) acc[e] += hand[q][lane * CPT + e];
      finish(k, acc);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------ small sort ---

// The whole sort in one launch, for up to kSmall positions whose key and
// position fit one word (key above, position below; no two are alike): a
// word's place is the number of words below it.  A workgroup has all words in
// LDS and ranks kRanked of them: lane l has word l % 16, and counts among four
// words at a time of its quarter of the wave's share.  The other workgroups of
// the launch clear dtable meanwhile.  N^2 comparisons, but spread over the
// device: a whole gradient of d = 250, V = 50021 takes 22 us at N = 4099, 28 at
// 8192 and 47 at 16384; with the radix sort's launches 34, 35 and 37.
constexpr int kSmall = 8192, kSmallThr = 1024, kRanked = 16;
__global__ void __launch_bounds__(kSmallThr) k_embed_rank(SortIn in, int N, int pos_bits, int n_rank,
                                                          uint32_t* __restrict__ keys, uint32_t* __restrict__ pos,
                                                          uint4* __restrict__ clear, int64_t n_clear,
                                                          uint8_t* __restrict__ tail, int n_tail) {
  constexpr int NW = kSmallThr / 64;
  __shared__ __attribute__((aligned(16))) uint32_t word[kSmall];
  __shared__ uint32_t below[NW][kRanked];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  if (static_cast<int>(blockIdx.x) >= n_rank) {
    const int64_t me = (static_cast<int64_t>(blockIdx.x) - n_rank) * kSmallThr + tid;
    const int64_t all = (static_cast<int64_t>(gridDim.x) - n_rank) * kSmallThr;
    for (int64_t i = me; i < n_clear; i += all) clear[i] = make_uint4(0, 0, 0, 0);
    if (me < n_tail) tail[me] = 0;
    return;
  }
  constexpr uint32_t kNone = 0xffffffffu;   // below no word
  const int quads = (N + 3) / 4;
  for (int i = tid; i < 4 * quads; i += kSmallThr)
    word[i] = i < N ? sort_key<true>(in, i) << pos_bits | static_cast<uint32_t>(i) : kNone;
  __syncthreads();
  const int at = static_cast<int>(blockIdx.x) * kRanked + lane % kRanked;
  const uint32_t mine = at < N ? word[at] : 0;
  uint32_t n = 0;
#pragma unroll 4
  for (int q = w * 4 + lane / kRanked; q < quads; q += 4 * NW) {
    const uint4 o = *reinterpret_cast<const uint4*>(word + 4 * q);
    n += (o.x < mine) + (o.y < mine) + (o.z < mine) + (o.w < mine);
  }
  n += __shfl_xor(n, 16, 64);
  n += __shfl_xor(n, 32, 64);
  if (lane < kRanked) below[w][lane] = n;
  __syncthreads();
  if (tid < kRanked && at < N) {
    uint32_t to = 0;
#pragma unroll
    for (int q = 0; q < NW; ++q) to += below[q][tid];
    keys[to] = mine >> pos_bits;
    pos[to] = static_cast<uint32_t>(at);
  }
}

// ----------------------------------------------------------------- host ---

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up(size_t x) { return (x + 255) / 256 * 256; }

// The tiles from which on their counts are summed up before the scatter: a whole
// gradient of d = 16, V = 50000 takes 112 us at 256 tiles (2048 tokens each)
// without and 143 with that, 226 and 239 at 512, 461 and 415 at 1024, 1051 and
// 763 at 2048.
constexpr int64_t kManyTiles = 640;

struct Plan {
  int key_bits, passes, bits, items;
  int64_t tiles, groups;
  size_t counts_off, sums_off, key_off[2], pos_off[2], part_off, total;
};
Plan plan(const EmbedArgs& a) {
  Plan p{};
  int bits = 1;
  while ((a.V >> bits) != 0) ++bits;   // keys 0 .. V
  p.key_bits = bits;
  p.passes = (bits + kMaxBits - 1) / kMaxBits;
  p.bits = (bits + p.passes - 1) / p.passes;
  // small tiles while they are few: every tile adds up the counts of all
  p.items = a.N <= 64 * 2 * kSortThr ? 2 : 4;
  p.tiles = cdiv(a.N, p.items * kSortThr);
  p.groups = p.tiles > kManyTiles ? cdiv(p.tiles, kGroup) : 0;
  size_t off = up(size_t(p.tiles) * kBins * 4);
  p.sums_off = off;
  if (p.groups) off += up(size_t(p.groups + 1) * kBins * 4);
  for (int i = 0; i < 2; ++i) {
    p.key_off[i] = off;
    off += up(size_t(a.N) * 4);
    p.pos_off[i] = off;
    off += up(size_t(a.N) * 4);
  }
  p.part_off = off;
  p.total = off + up(2 * size_t(cdiv(a.N, kBlock)) * a.d * 4);
  return p;
}

// are they sorted in one launch?
bool small_sort(const EmbedArgs& a, int key_bits, int* pos_bits) {
  int pb = 1;
  while (((a.N - 1) >> pb) != 0) ++pb;
  *pos_bits = pb;
  return a.N <= kSmall && key_bits + pb <= 32;
}

template <int DT, int VEC>
void embed_vec(const EmbedArgs& a, const void* tokens, const void* table, void* out) {
  using T = typename Storage<DT>::T;
  auto run = [&](auto tpr) {
    constexpr int TPR = decltype(tpr)::value;
    k_embed<DT, VEC, TPR><<<rows_of_blocks(cdiv(a.N, 256 / TPR * kRows)), 256, 0, a.stream>>>(
        tokens, a.token_bytes, static_cast<const T*>(table), a.N, a.V, a.d, a.scale, a.pad, static_cast<T*>(out));
  };
  if (a.d <= 16 * VEC) run(std::integral_constant<int, 16>{});
  else run(std::integral_constant<int, 64>{});
}

template <int DT, int VEC>
void sum_vec(const EmbedArgs& a, const Plan& p, const uint32_t* keys, const uint32_t* pos, const void* dout, void* dtable) {
  using T = typename Storage<DT>::T;
  constexpr int CPT = VEC > 4 ? 4 : VEC;
  float* part = reinterpret_cast<float*>(a.ws + p.part_off);
  const dim3 grid = rows_of_blocks(cdiv(cdiv(a.N, kBlock), 4), cdiv(a.d, 64 * VEC));
  k_embed_sum<DT, VEC><<<grid, 256, 0, a.stream>>>(keys, pos, static_cast<const T*>(dout), a.N, a.V, a.d, a.scale,
                                                   static_cast<T*>(dtable), part);
  if (a.N < kLong) return;
  const dim3 jgrid = rows_of_blocks(cdiv(a.N, kJoin), cdiv(a.d, 64 * CPT));
  k_embed_join<DT, CPT><<<jgrid, kJoinThr, 0, a.stream>>>(keys, part, a.N, a.V, a.d, a.scale, static_cast<T*>(dtable));
}

}  // namespace

size_t embed_backward_workspace(const EmbedArgs& a) { return a.N ? plan(a).total : 0; }

void launch_embed(const EmbedArgs& a, const void* tokens, const void* table, void* out) {
  if (a.bf16)
    return a.d >= kVec<kBF16> ? embed_vec<kBF16, kVec<kBF16>>(a, tokens, table, out) : embed_vec<kBF16, 1>(a, tokens, table, out);
  return a.d >= kVec<kF32> ? embed_vec<kF32, kVec<kF32>>(a, tokens, table, out) : embed_vec<kF32, 1>(a, tokens, table, out);
}

void launch_embed_backward(const EmbedArgs& a, const void* tokens, const void* dout, void* dtable) {
  const Plan p = plan(a);
  uint32_t* counts = reinterpret_cast<uint32_t*>(a.ws + p.counts_off);
  uint32_t* sums = reinterpret_cast<uint32_t*>(a.ws + p.sums_off);
  uint32_t *keys[2], *pos[2];
  for (int i = 0; i < 2; ++i) {
    keys[i] = reinterpret_cast<uint32_t*>(a.ws + p.key_off[i]);
    pos[i] = reinterpret_cast<uint32_t*>(a.ws + p.pos_off[i]);
  }
  const size_t bytes = size_t(a.V) * a.d * (a.bf16 ? 2 : 4);
  uint8_t* const lo = static_cast<uint8_t*>(dtable);   // 16-byte aligned
  const int64_t words = int64_t(bytes / 16);
  uint4* const clear = reinterpret_cast<uint4*>(lo);
  uint8_t* const tail = lo + words * 16;
  const int n_tail = int(bytes % 16);
  SortIn in{tokens, a.token_bytes, a.V, a.pad, nullptr, nullptr};
  int cur = 0, pos_bits;
  if (a.N > 0 && small_sort(a, p.key_bits, &pos_bits)) {
    const unsigned ranks = unsigned(cdiv(a.N, kRanked)), others = unsigned(std::min<int64_t>(512, cdiv(words, kSmallThr) + 1));
    k_embed_rank<<<ranks + others, kSmallThr, 0, a.stream>>>(in, int(a.N), pos_bits, int(ranks), keys[0], pos[0], clear, words,
                                                             tail, n_tail);
  } else {
    auto sort = [&](auto items) {
      constexpr int IT = decltype(items)::value;
      const unsigned tiles = unsigned(p.tiles), others = unsigned(std::min<int64_t>(1024, cdiv(words, kSortThr) + 1));
      const int groups = int(p.groups);
      auto offsets = [&]() {
        if (!groups) return;
        k_embed_offsets<<<unsigned(groups), kSortThr, 0, a.stream>>>(counts, int(tiles), kGroup, sums);
        k_embed_offsets<<<1, kSortThr, 0, a.stream>>>(sums, groups, groups, sums + int64_t(groups) * kBins);
      };
      for (int s = 0; s < p.passes; ++s) {
        const int shift = s * p.bits;
        if (s == 0) {
          k_embed_count<true, IT><<<tiles + others, kSortThr, 0, a.stream>>>(in, a.N, shift, p.bits, int(tiles), counts,
                                                                             clear, words, tail, n_tail);
          if (a.N == 0) return;
          offsets();
          k_embed_scatter<true, IT><<<tiles, kSortThr, 0, a.stream>>>(in, a.N, shift, p.bits, int(tiles), counts, sums, groups,
                                                                      keys[0], pos[0]);
          continue;
        }
        in.keys = keys[cur];
        in.pos = pos[cur];
        k_embed_count<false, IT><<<tiles, kSortThr, 0, a.stream>>>(in, a.N, shift, p.bits, int(tiles), counts, nullptr, 0,
                                                                   nullptr, 0);
        offsets();
        k_embed_scatter<false, IT><<<tiles, kSortThr, 0, a.stream>>>(in, a.N, shift, p.bits, int(tiles), counts, sums, groups,
                                                                     keys[cur ^ 1], pos[cur ^ 1]);
        cur ^= 1;
      }
    };
    if (p.items == 2) sort(std::integral_constant<int, 2>{}); else sort(std::integral_constant<int, 4>{});
    if (a.N == 0) return;
  }
  if (a.bf16) {
    if (a.d >= kVec<kBF16>) return sum_vec<kBF16, kVec<kBF16>>(a, p, keys[cur], pos[cur], dout, dtable);
    return sum_vec<kBF16, 1>(a, p, keys[cur], pos[cur], dout, dtable);
  }
  if (a.d >= kVec<kF32>) return sum_vec<kF32, kVec<kF32>>(a, p, keys[cur], pos[cur], dout, dtable);
  return sum_vec<kF32, 1>(a, p, keys[cur], pos[cur], dout, dtable);
}

}  // namespace prn
