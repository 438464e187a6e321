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

#include "prn_device.h"

namespace prn {
namespace {

constexpr int kTile = 2048;     // positions a workgroup sorts
constexpr int kSortThr = 256;
constexpr int kItems = kTile / kSortThr;
constexpr int kMaxBits = 9;     // of a radix pass
constexpr int kBins = 1 << kMaxBits;
constexpr int kBlock = 16;      // sorted positions a group of lanes starts from
constexpr int kLong = 64;       // rows of a chunk of a frequent token (a multiple of kBlock)

template <int DT, int VEC> struct Pack;
template <> struct Pack<kF32, 4> { using T = uint4; };
template <> struct Pack<kF32, 2> { using T = uint2; };
template <> struct Pack<kF32, 1> { using T = uint32_t; };
template <> struct Pack<kBF16, 8> { using T = uint4; };
template <> struct Pack<kBF16, 4> { using T = uint2; };
template <> struct Pack<kBF16, 2> { using T = uint32_t; };
template <> struct Pack<kBF16, 1> { using T = uint16_t; };

template <int DT, int VEC>
__device__ __forceinline__ void load_vec(const typename Storage<DT>::T* p, float* o) {
  using P = typename Pack<DT, VEC>::T;
  const P q = *reinterpret_cast<const P*>(p);
  typename Storage<DT>::T t[VEC];
  __builtin_memcpy(t, &q, sizeof(q));
#pragma unroll
  for (int e = 0; e < VEC; ++e) o[e] = Storage<DT>::load(&t[e]);
}
template <int DT, int VEC>
__device__ __forceinline__ void store_vec(typename Storage<DT>::T* p, const float* o) {
  using P = typename Pack<DT, VEC>::T;
  typename Storage<DT>::T t[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) t[e] = Storage<DT>::pack(o[e]);
  P q;
  __builtin_memcpy(&q, t, sizeof(q));
  *reinterpret_cast<P*>(p) = q;
}

__device__ __forceinline__ int64_t token_at(const void* tokens, int bytes, int64_t n) {
  return bytes == 4 ? static_cast<int64_t>(static_cast<const int32_t*>(tokens)[n])
                    : static_cast<const int64_t*>(tokens)[n];
}

// TPR lanes per row.  The pad token's rows are zeros, a token outside the
// table gives NaN.
template <int DT, int VEC, int TPR>
__global__ void __launch_bounds__(256) k_embed(const void* __restrict__ tokens, int token_bytes,
                                               const typename Storage<DT>::T* __restrict__ table, int64_t N, int64_t V,
                                               int64_t d, float scale, int64_t pad,
                                               typename Storage<DT>::T* __restrict__ out) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * (256 / TPR) + threadIdx.x / TPR;
  if (n >= N) return;
  const int64_t t = token_at(tokens, token_bytes, n);
  const bool in = t >= 0 && t < V && t != pad;
  const float fill = t == pad ? 0.0f : __builtin_nanf("");
  const typename Storage<DT>::T* src = table + (in ? t : 0) * d;
  for (int64_t c = static_cast<int64_t>(threadIdx.x % TPR) * VEC; c < d; c += TPR * VEC) {
    float v[VEC];
    load_vec<DT, VEC>(src + c, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = in ? v[e] * scale : fill;
    store_vec<DT, VEC>(out + n * d + c, v);
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
template <bool FIRST>
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
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kTile;
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const int64_t i = at + j * kSortThr + threadIdx.x;
    if (i < N) atomicAdd(&hist[(sort_key<FIRST>(in, i) >> shift) & ((1u << bits) - 1)], 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < (1 << bits); b += kSortThr)
    counts[static_cast<int64_t>(blockIdx.x) * kBins + b] = hist[b];
}

// Stable scatter by one digit: wave w of a tile holds its positions 512 w ..
// + 511 in order; a position's rank among the equal digits before it in the
// wave comes from ballots, the counts of earlier waves, tiles and digits are
// added to it.
template <bool FIRST>
__global__ void __launch_bounds__(kSortThr) k_embed_scatter(SortIn in, int64_t N, int shift, int bits, int n_tiles,
                                                            const uint32_t* __restrict__ counts,
                                                            uint32_t* __restrict__ keys_out,
                                                            uint32_t* __restrict__ pos_out) {
  constexpr int NW = kSortThr / 64;
  __shared__ uint32_t start[kBins];        // where the tile's first position of a digit goes
  __shared__ uint32_t wave_hist[NW][kBins];
  __shared__ uint32_t scan[NW];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int nb = 1 << bits;
  for (int b = lane; b < nb; b += 64) wave_hist[w][b] = 0;
  __syncthreads();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kTile + w * (kTile / NW);
  // other lanes of the wave write it between two reads
  volatile uint32_t* const mine_hist = wave_hist[w];
  uint32_t key[kItems], pos[kItems], rank[kItems];
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const int64_t i = at + j * 64 + lane;
    key[j] = i < N ? sort_key<FIRST>(in, i) : 0;
    pos[j] = FIRST ? static_cast<uint32_t>(i) : i < N ? in.pos[i] : 0;
  }
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const bool live = at + j * 64 + lane < N;
    const uint32_t dg = (key[j] >> shift) & (nb - 1);
    unsigned long long same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
      const unsigned long long m = __ballot((dg >> b) & 1);
      same &= (dg >> b) & 1 ? m : ~m;
    }
    if (live) {
      const unsigned long long below = same & ((1ull << lane) - 1);
      const uint32_t before = mine_hist[dg];
      rank[j] = before + __popcll(below);
      // the last lane of the digit counts them all (a wave's LDS accesses are done in order)
      if ((same >> lane) == 1ull) mine_hist[dg] = before + __popcll(same);
    }
  }
  // digit totals, and those of the tiles before this one
  uint32_t total[kBins / kSortThr], before[kBins / kSortThr];
#pragma unroll
  for (int q = 0; q < kBins / kSortThr; ++q) {
    const int b = 2 * tid + q;
    uint32_t all = 0, less = 0;
    if (b < nb) {
#pragma unroll 8
      for (int t = 0; t < n_tiles; ++t) {
        const uint32_t c = counts[static_cast<int64_t>(t) * kBins + b];
        all += c;
        less += t < static_cast<int>(blockIdx.x) ? c : 0;
      }
    }
    total[q] = all;
    before[q] = less;
  }
  // exclusive sum of the totals over the digits (two neighbouring digits a thread)
  const uint32_t mine = total[0] + total[1];
  uint32_t incl = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = __shfl_up(incl, o, 64);
    if (lane >= o) incl += up;
  }
  if (lane == 63) scan[w] = incl;
  __syncthreads();   // also: every wave's histogram is complete
  uint32_t base = incl - mine;
  for (int q = 0; q < w; ++q) base += scan[q];
  start[2 * tid] = base + before[0];
  start[2 * tid + 1] = base + total[0] + before[1];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    if (at + j * 64 + lane < N) {
      const uint32_t dg = (key[j] >> shift) & (nb - 1);
      uint32_t to = start[dg] + rank[j];
      for (int q = 0; q < w; ++q) to += wave_hist[q][dg];
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
    float v[kBatch][VEC];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      if (i + q < i1 && mine) load_vec<DT, VEC>(dout + static_cast<int64_t>(where(i + q)) * d + c, v[q]);
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      if (i + q < i1) {
        emit(i + q, acc);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += v[q][e];
      }
    }
  }
}

// A wave per kBlock sorted positions and 64 VEC channels (blockIdx.y): sums
// every token whose rows start there, and the chunk of a frequent token from
// an earlier block that starts there (at most one: chunks are kLong >= kBlock
// apart).  A frequent token's chunks go to part: its first to row 2 block + 1,
// the others to row 2 block.  The keys and positions of the 127 sorted places
// a wave may need are loaded at once; every decision after that is a ballot.
template <int DT, int VEC>
__global__ void __launch_bounds__(256) k_embed_sum(const uint32_t* __restrict__ keys, const uint32_t* __restrict__ pos,
                                                   const typename Storage<DT>::T* __restrict__ dout, int64_t N, int64_t V,
                                                   int64_t d, float scale, typename Storage<DT>::T* __restrict__ dtable,
                                                   float* __restrict__ part) {
  constexpr uint32_t kNone = 0xffffffffu;   // above every key
  const int lane = threadIdx.x & 63;
  const int64_t block = static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t p0 = block * kBlock;
  if (p0 >= N) return;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * 64 + lane) * VEC;
  const bool mine = c < d;
  // place t (position p0 + t): lane t + 1 of the first window for t < 63, lane t - 63 of the second
  const int64_t ia = p0 - 1 + lane, ib = p0 + 63 + lane;
  const uint32_t ka = ia >= 0 && ia < N ? keys[ia] : kNone, kb = ib < N ? keys[ib] : kNone;
  const uint32_t qa = ia >= 0 && ia < N ? pos[ia] : 0, qb = ib < N ? pos[ib] : 0;
  const uint32_t prev_a = __shfl_up(ka, 1, 64), last_a = __shfl(ka, 63, 64), prev_b = __shfl_up(kb, 1, 64);
  const uint32_t kb_at = __shfl_up(kb, 1, 64);   // lane t + 1: the key kLong - 1 places after place t
  // bit t: place t holds another key than place t - 1; bit l of the second: place 63 + l
  const unsigned long long turn_a = __ballot(lane >= 1 && ka != prev_a) >> 1;
  const unsigned long long turn_b = __ballot(kb != (lane == 0 ? last_a : prev_b));
  const unsigned own = static_cast<unsigned>(turn_a & __ballot(ka < V) >> 1) & ((1u << kBlock) - 1);
  const unsigned frequent = own & static_cast<unsigned>(__ballot(ka == kb_at) >> 1);
  float acc[VEC];
  auto to_part = [&](int64_t row) {
    if (mine) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) part[row * d + c + e] = acc[e];
    }
  };

  const uint32_t k0 = __shfl(ka, 1, 64);
  if (!(turn_a & 1) && k0 < V) {
    // a token from an earlier block: its chunk that starts here, if it is a frequent one
    const int64_t s = lower_bound(keys, p0, k0);
    if (s + kLong <= N && keys[s + kLong - 1] == k0) {
      const int64_t b = s + (p0 - s + kLong - 1) / kLong * kLong;
      const unsigned long long run = __ballot(b + lane < N && keys[b + lane < N ? b + lane : N - 1] == k0);
      const uint32_t at = b + lane < N ? pos[b + lane] : 0;
      if (b < p0 + kBlock && (run & 1)) {
        const int n = ~run == 0 ? 64 : __builtin_ctzll(~run);
        walk_rows<DT, VEC>(dout, d, c, mine, 0, n, [&](int i) { return __builtin_amdgcn_readlane(at, i); },
                           [](int, float*) {}, acc);
        to_part(2 * block);
      }
    }
  }
  if (!own) return;
  const int t0 = __builtin_ctz(own), t1 = 31 - __builtin_clz(own);   // first and last token that starts here
  const bool last_frequent = (frequent >> t1) & 1;
  const unsigned long long rest = turn_a >> (t1 + 1);
  // the next turn, in the first window or (a shorter run ends by place t1 + kLong - 1) the second
  const int end = last_frequent ? t1 + kLong : rest ? t1 + 1 + __builtin_ctzll(rest) : 63 + __builtin_ctzll(turn_b);
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
      [&](int t) { return t < 63 ? __builtin_amdgcn_readlane(qa, t + 1) : __builtin_amdgcn_readlane(qb, t - 63); },
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
// sums, added in order by 16 waves (every 16th chunk each, then the waves in
// order), 64 channels at a time.
constexpr int kJoin = 1024;
template <int DT>
__global__ void __launch_bounds__(1024) k_embed_join(const uint32_t* __restrict__ keys, const float* __restrict__ part,
                                                     int64_t N, int64_t V, int64_t d, float scale,
                                                     typename Storage<DT>::T* __restrict__ dtable) {
  __shared__ uint32_t n_found;
  __shared__ uint32_t found[kJoin / kLong + 1];
  __shared__ float hand[16][64];
  if (threadIdx.x == 0) n_found = 0;
  __syncthreads();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kJoin;
  const int64_t p = at + threadIdx.x;
  if (p + kLong <= N) {
    const uint32_t k = keys[p];
    if (k < V && keys[p + kLong - 1] == k && (p == 0 || keys[p - 1] != k)) found[atomicAdd(&n_found, 1u)] = threadIdx.x;
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (uint32_t f = 0; f < n_found; ++f) {   // in any order: each writes its own row
    const int64_t s = at + found[f];
    const uint32_t k = keys[s];
    const int64_t len = lower_bound(keys, N, k + 1) - s, chunks = (len + kLong - 1) / kLong;
    for (int64_t c0 = 0; c0 < d; c0 += 64) {
      const int64_t c = c0 + lane;
      float acc = 0.0f;
      if (c < d) {
#pragma unroll 4
        for (int64_t q = w; q < chunks; q += 16) acc += part[(2 * ((s + q * kLong) / kBlock) + (q == 0)) * d + c];
      }
      hand[w][lane] = acc;
      __syncthreads();
      if (w == 0 && c < d) {
#pragma unroll
        for (int q = 1; q < 16; ++q) acc += hand[q][lane];
        dtable[static_cast<int64_t>(k) * d + c] = Storage<DT>::pack(acc * scale);
      }
      __syncthreads();
    }
  }
}

// ----------------------------------------------------------------- host ---

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up(size_t x) { return (x + 255) / 256 * 256; }

struct Plan {
  int passes, bits;
  int64_t tiles;
  size_t counts_off, key_off[2], pos_off[2], part_off, total;
};
Plan plan(const EmbedArgs& a) {
  Plan p{};
  int bits = 1;
  while ((a.V >> bits) != 0) ++bits;   // keys 0 .. V
  p.passes = (bits + kMaxBits - 1) / kMaxBits;
  p.bits = (bits + p.passes - 1) / p.passes;
  p.tiles = cdiv(a.N, kTile);
  size_t off = up(size_t(p.tiles) * kBins * 4);
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

// elements per access: the largest power of two that divides a row and its
// 16 bytes and keeps every base aligned
int vec_of(bool bf16, int64_t d, const void* p, const void* q) {
  const int elt = bf16 ? 2 : 4;
  int v = 16 / elt;
  while (v > 1 && (d % v != 0 || reinterpret_cast<uintptr_t>(p) % (v * elt) != 0 ||
                   reinterpret_cast<uintptr_t>(q) % (v * elt) != 0))
    v /= 2;
  return v;
}

template <int DT, int VEC>
void embed_vec(const EmbedArgs& a, const void* tokens, const void* table, void* out) {
  using T = typename Storage<DT>::T;
  auto run = [&](auto tpr) {
    constexpr int TPR = decltype(tpr)::value;
    k_embed<DT, VEC, TPR><<<unsigned(cdiv(a.N, 256 / TPR)), 256, 0, a.stream>>>(
        tokens, a.token_bytes, static_cast<const T*>(table), a.N, a.V, a.d, a.scale, a.pad, static_cast<T*>(out));
  };
  if (a.d <= 16 * VEC) run(std::integral_constant<int, 16>{});
  else run(std::integral_constant<int, 64>{});
}

template <int DT, int VEC>
void sum_vec(const EmbedArgs& a, const Plan& p, const uint32_t* keys, const uint32_t* pos, const void* dout, void* dtable) {
  using T = typename Storage<DT>::T;
  float* part = reinterpret_cast<float*>(a.ws + p.part_off);
  const dim3 grid(unsigned(cdiv(cdiv(a.N, kBlock), 4)), unsigned(cdiv(a.d, 64 * VEC)));
  k_embed_sum<DT, VEC><<<grid, 256, 0, a.stream>>>(keys, pos, static_cast<const T*>(dout), a.N, a.V, a.d, a.scale,
                                                   static_cast<T*>(dtable), part);
  k_embed_join<DT><<<unsigned(cdiv(a.N, kJoin)), 1024, 0, a.stream>>>(keys, part, a.N, a.V, a.d, a.scale,
                                                                       static_cast<T*>(dtable));
}

}  // namespace

size_t embed_backward_workspace(const EmbedArgs& a) { return a.N ? plan(a).total : 0; }

void launch_embed(const EmbedArgs& a, const void* tokens, const void* table, void* out) {
  const int v = vec_of(a.bf16, a.d, table, out);
  if (a.bf16) {
    if (v == 8) return embed_vec<kBF16, 8>(a, tokens, table, out);
    if (v == 4) return embed_vec<kBF16, 4>(a, tokens, table, out);
    if (v == 2) return embed_vec<kBF16, 2>(a, tokens, table, out);
    return embed_vec<kBF16, 1>(a, tokens, table, out);
  }
  if (v == 4) return embed_vec<kF32, 4>(a, tokens, table, out);
  if (v == 2) return embed_vec<kF32, 2>(a, tokens, table, out);
  return embed_vec<kF32, 1>(a, tokens, table, out);
}

void launch_embed_backward(const EmbedArgs& a, const void* tokens, const void* dout, void* dtable) {
  const Plan p = plan(a);
  uint32_t* counts = reinterpret_cast<uint32_t*>(a.ws + p.counts_off);
  uint32_t *keys[2], *pos[2];
  for (int i = 0; i < 2; ++i) {
    keys[i] = reinterpret_cast<uint32_t*>(a.ws + p.key_off[i]);
    pos[i] = reinterpret_cast<uint32_t*>(a.ws + p.pos_off[i]);
  }
  const size_t bytes = size_t(a.V) * a.d * (a.bf16 ? 2 : 4);
  uint8_t* const lo = static_cast<uint8_t*>(dtable);   // 16-byte aligned
  const int64_t words = int64_t(bytes / 16);
  SortIn in{tokens, a.token_bytes, a.V, a.pad, nullptr, nullptr};
  int cur = 0;
  for (int s = 0; s < p.passes; ++s) {
    const int shift = s * p.bits;
    const unsigned tiles = unsigned(p.tiles);
    if (s == 0) {
      const unsigned clear = unsigned(std::min<int64_t>(1024, cdiv(words, kSortThr) + 1));
      k_embed_count<true><<<tiles + clear, kSortThr, 0, a.stream>>>(in, a.N, shift, p.bits, int(tiles), counts,
                                                                    reinterpret_cast<uint4*>(lo), words, lo + words * 16,
                                                                    int(bytes % 16));
      if (a.N == 0) return;
      k_embed_scatter<true><<<tiles, kSortThr, 0, a.stream>>>(in, a.N, shift, p.bits, int(tiles), counts, keys[0], pos[0]);
    } else {
      in.keys = keys[cur];
      in.pos = pos[cur];
      k_embed_count<false><<<tiles, kSortThr, 0, a.stream>>>(in, a.N, shift, p.bits, int(tiles), counts, nullptr, 0, nullptr, 0);
      k_embed_scatter<false><<<tiles, kSortThr, 0, a.stream>>>(in, a.N, shift, p.bits, int(tiles), counts, keys[cur ^ 1],
                                                               pos[cur ^ 1]);
      cur ^= 1;
    }
  }
  const int v = vec_of(a.bf16, a.d, dout, dtable);
  if (a.bf16) {
    if (v == 8) return sum_vec<kBF16, 8>(a, p, keys[cur], pos[cur], dout, dtable);
    if (v == 4) return sum_vec<kBF16, 4>(a, p, keys[cur], pos[cur], dout, dtable);
    if (v == 2) return sum_vec<kBF16, 2>(a, p, keys[cur], pos[cur], dout, dtable);
    return sum_vec<kBF16, 1>(a, p, keys[cur], pos[cur], dout, dtable);
  }
  if (v == 4) return sum_vec<kF32, 4>(a, p, keys[cur], pos[cur], dout, dtable);
  if (v == 2) return sum_vec<kF32, 2>(a, p, keys[cur], pos[cur], dout, dtable);
  return sum_vec<kF32, 1>(a, p, keys[cur], pos[cur], dout, dtable);
}

}  // namespace prn
