// Matrix-core tiles over bf16 or fp16 operands of either orientation, for the
// vocabulary loss: acc = sum over k of A(r, k) B(c, k).
//
// Each wave owns WM x WN blocks of 32 x 32; WR x WC waves make a workgroup's
// tile of BM x BN.  K is walked in stages of BK values, NST stages in LDS,
// the next ones in flight while one is multiplied.  An operand lies in memory
// as rows of K ("rows": element (r, k) at r ld + k) or as rows of the other
// index ("cols": element (r, k) at k ld + r); neither is transposed or copied
// on the way: both land in LDS as they are, and the "cols" fragments come
// through ds_read_b64_tr_b16.
//
// Loads go straight into LDS (global_load_lds_dwordx4: lane l of a wave's
// load lands at LDS base + 16 l), 1 KB a wave load.  In LDS the 16-byte
// chunks of a row are permuted, so that the rows one fragment read touches
// fall on all banks:
//   rows: BK = 64: 128-byte rows, chunk c of row r at c ^ ((r / 2) % 8);
//         BK = 32: 64-byte rows, chunk c at c ^ ((r / 4) % 4)
//   cols: rows of 2 BM bytes, chunk c of row k at c ^ swz(k); swz keeps the
//         eight rows of one transposed read (k0 .. k0 + 3 and k0 + 8 ..
//         k0 + 11) on different banks.
// A wait for a wave's own loads and a bare barrier make a stage complete (a
// fence would drain the stages still in flight too).  They come before a
// stage's last 16 k: its fragments are in registers by then, so its buffer is
// free for the next load, and the next stage's first fragments are read while
// the last products run.  (With the wait at the head of a stage the cores
// stood still for it and the reads behind it: the logits of 32768 x 512 x 32768
// took 1.17 ms, now 1.05.)
// What bounds it: the energy of a product.  At 256 x 256 the loop runs at 1.0 ..
// 1.15 PFLOP/s of random data (the matrix cores busy 53 .. 60% of the cycles, at
// 1.85 GHz of 2.4) and at 1.76 of zeros; a library product of 8192^3, with longer
// sums and wider waves, has 1.45 under the same power.
//
// Fragment layout of v_mfma_f32_32x32x16_bf16 and _f16: lane l feeds row l % 32 of A
// and column l % 32 of B with the k values 8 (l / 32) .. + 7; accumulator r
// of lane l holds row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace prn {

typedef __attribute__((ext_vector_type(8))) __bf16 mm_bf16x8;
typedef __attribute__((ext_vector_type(2))) _Float16 mm_f16x2;
typedef __attribute__((ext_vector_type(8))) _Float16 mm_f16x8;
typedef __attribute__((ext_vector_type(16))) float mm_f32x16;
typedef __attribute__((ext_vector_type(4))) short mm_s16x4;
typedef __attribute__((ext_vector_type(8))) short mm_s16x8;
typedef __attribute__((ext_vector_type(4))) uint32_t mm_u32x4;
typedef __attribute__((address_space(3))) void* mm_lds_t;

__device__ __attribute__((aligned(16))) const uint32_t kMmZero[4] = {0, 0, 0, 0};

__device__ __forceinline__ uint32_t mm_lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((mm_lds_t) const_cast<void*>(p)));
}

// One direct-to-LDS load of 16 bytes per lane to LDS byte lds + 16 lane (lds
// wave-uniform, through M0, which nothing else here uses; one wait state
// between the scalar write of M0 and its use).  In asm, so that the compiler
// does not make every later LDS read wait for it; the stage loop waits.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // M0 is a reserved register
__device__ __forceinline__ void mm_dma(const void* g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(g), "s"(lds) : "memory", "m0");
}
// a wave-uniform pointer in scalar registers
__device__ __forceinline__ const void* mm_uniform(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const void*>(static_cast<uint64_t>(hi) << 32 | lo);
}
// the load from a wave-uniform base and a byte offset per lane
__device__ __forceinline__ void mm_dma_off(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// wait until at most n of this wave's loads are in flight, and for all its LDS reads
template <int n>
__device__ __forceinline__ void mm_wait_loads() {
  static_assert(n >= 0 && n <= 63, "six bits of the load counter, in two places");
  __builtin_amdgcn_s_waitcnt((n & 15) | (7 << 4) | ((n >> 4) << 14));
}

// one product of two fragments of bf16 or fp16 values
template <bool F16>
__device__ __forceinline__ mm_f32x16 mm_product(mm_bf16x8 a, mm_bf16x8 b, mm_f32x16 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(mm_f16x8, a), __builtin_bit_cast(mm_f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// An operand: a 16-bit matrix, rows ld elements apart, ld a multiple of 8, base
// 16-byte aligned.  Along its contiguous index the memory holds a multiple of 8
// values per row (the ones past the extent are zeros where that index is k,
// anything otherwise).  Of two-term data (PAIR) every 32 values along that
// index are 64: the 32 high terms, then the 32 low ones.
struct MmOperand {
  const uint16_t* base;
  int64_t ld;
};

// PAIR: two-term operands.  A stage holds both terms of BK / 2 = 32 values of
// k, the high ones in the first half of its k places; the product takes high
// high, high low and low high (the low terms' own product is left out).  Every
// term is loaded and read once for its two products, where a pass per pair of
// terms loads and reads half as much again (4096 x 256 x 32000, each way: 955
// us; this takes 860).
template <int WR_, int WC_, int WM_, int WN_, int BK_, int NST_, bool PAIR_ = false>
struct MmTile {
  static constexpr int WR = WR_, WC = WC_, WM = WM_, WN = WN_, BK = BK_, NST = NST_;
  static constexpr bool PAIR = PAIR_;
  static constexpr int KS = PAIR ? BK / 2 : BK;   // k of a stage
  static_assert(!PAIR || BK == 64, "32 and 32");
  static constexpr int NW = WR * WC, NTHR = 64 * NW;
  static constexpr int BM = WR * WM * 32, BN = WC * WN * 32;
  static constexpr int ABYTES = BM * BK * 2, BBYTES = BN * BK * 2, STAGE = ABYTES + BBYTES;
  static constexpr int LDS = NST * STAGE;
  static constexpr int NLA = ABYTES / 1024 / NW, NLB = BBYTES / 1024 / NW;   // wave loads of a wave per stage
  static_assert(ABYTES % (1024 * NW) == 0 && BBYTES % (1024 * NW) == 0, "stages split evenly over the waves");
  static_assert(BK == 32 || BK == 64, "row layouts of 64 and 128 bytes");
  static_assert((NST - 2) * (NLA + NLB) <= 63, "load counter");

  mm_f32x16 acc[WM][WN];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < WM; ++i)
#pragma unroll
      for (int j = 0; j < WN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  }

  static __device__ __forceinline__ int row_pos(int r, int c) {
    return BK == 64 ? c ^ ((r >> 1) & 7) : c ^ ((r >> 2) & 3);
  }
  // where the chunks of row k (of CPR) go: c ^ swz
  template <int CPR>
  static __device__ __forceinline__ int swz(int k) {
    static_assert(CPR == 24 || (CPR & (CPR - 1)) == 0, "XOR stays within a row");
    if constexpr (CPR == 24)
      return 4 * ((k >> 1) & 1);   // rows of 384 bytes: neighbours are half of the banks apart by themselves
    else
      return 4 * ((k & 3) | (((k >> 3) & 1) << 2)) & (CPR - 1);
  }

  // lane's source chunk of wave load li of an operand with BR rows of the
  // tile index: (row or k within the stage, first element along the contiguous index)
  template <bool COLS, int BR>
  static __device__ __forceinline__ void source(int li, int lane, int& slow, int& fast) {
    const int v = li * 64 + lane;
    if constexpr (!COLS) {
      constexpr int CPR = BK / 8;
      slow = v / CPR;
      fast = 8 * row_pos(slow, v % CPR);
    } else {
      constexpr int CPR = BR / 8;
      slow = v / CPR;
      fast = 8 * ((v % CPR) ^ swz<CPR>(slow));
    }
  }

  // The stream of stages: tile after tile, each k0 .. k1.
  // The loads run NST - 1 stages ahead of the products, across tiles too, so
  // that the next tile's first stages are in flight during an epilogue.
  uint8_t* lds;
  MmOperand A, B;
  int64_t Ra, Rb, k0, k1;   // rows of the operands in all; the summed range (k0 a multiple of 8, PAIR: 32)
  int nk, nfull, ntail;     // stages, full ones, the last one's blocks of 16 k
  uint32_t offa[NLA], offb[NLB];
  const uint8_t *ab, *bb;
  int at_k;                 // the next stage to load
  bool more;                // there is one
  int ahead;                // stages loaded and not yet multiplied
  int buf_load, buf_use;

  __device__ __forceinline__ void open(uint8_t* lds_, const MmOperand& A_, int64_t Ra_, const MmOperand& B_, int64_t Rb_,
                                       int64_t k0_, int64_t k1_) {
    lds = lds_, A = A_, B = B_, Ra = Ra_, Rb = Rb_, k0 = k0_, k1 = k1_;
    nk = k1 > k0 ? static_cast<int>((k1 - k0 + KS - 1) / KS) : 0;
    nfull = k1 > k0 ? static_cast<int>((k1 - k0) / KS) : 0;
    ntail = nk > 0 ? static_cast<int>((k1 - k0 - static_cast<int64_t>(nk - 1) * KS + 15) / 16) : 0;
    more = false;
    ahead = buf_load = buf_use = 0;
  }

  // the next tile to load: rows r0 .. of A, c0 .. of B
  template <bool TA, bool TB>
  __device__ __forceinline__ void seek(int64_t r0, int64_t c0) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    offsets<TA, BM, NLA>(wave, lane, A.ld, Ra, r0, offa);
    offsets<TB, BN, NLB>(wave, lane, B.ld, Rb, c0, offb);
    constexpr int F = PAIR ? 2 : 1;
    ab = reinterpret_cast<const uint8_t*>(A.base + (TA ? k0 * A.ld + F * r0 : r0 * A.ld + F * k0));
    bb = reinterpret_cast<const uint8_t*>(B.base + (TB ? k0 * B.ld + F * c0 : c0 * B.ld + F * k0));
    at_k = 0;
    more = nk > 0;
  }

  // Byte offsets of a wave's loads from the tile's first element.  Rows past
  // the end read the last row, columns past the end the last chunk: what
  // comes of them is not used.
  template <bool COLS, int BR, int NL>
  static __device__ __forceinline__ void offsets(int wave, int lane, int64_t ld, int64_t R, int64_t r0, uint32_t (&off)[NL]) {
    const int64_t left = COLS ? ((R + 7) & ~int64_t(7)) - 8 - r0 : R - 1 - r0;
    const int lim = left < BR ? static_cast<int>(left) : BR;
#pragma unroll
    for (int p = 0; p < NL; ++p) {
      int s, f;
      source<COLS, BR>(wave * NL + p, lane, s, f);
      if constexpr (COLS) f = f < lim ? f : lim; else s = s < lim ? s : lim;
      if constexpr (COLS && PAIR) {
        f = 2 * (f & ~31) + (f & 31) + 32 * (s / KS);
        s %= KS;
      }
      off[p] = static_cast<uint32_t>((s * ld + f) * 2);
    }
  }
  // One operand's loads of a stage.  In the last, partial stage (left < KS
  // values of k) the chunks past the end come from the zero chunk.
  template <bool COLS, int BR, int NL>
  static __device__ __forceinline__ void load_operand(const uint8_t* base, const uint32_t (&off)[NL], uint8_t* dst, int wave,
                                                      int left) {
    if (left >= KS) {
#pragma unroll
      for (int p = 0; p < NL; ++p) mm_dma_off(mm_uniform(base), off[p], mm_lds_addr(dst + p * 1024));
    } else {
      const int lane = threadIdx.x & 63;
#pragma unroll
      for (int p = 0; p < NL; ++p) {
        int s, f;
        source<COLS, BR>(wave * NL + p, lane, s, f);
        const void* g = (COLS ? s : f) % KS < left ? static_cast<const void*>(base + off[p]) : static_cast<const void*>(kMmZero);
        mm_dma(g, mm_lds_addr(dst + p * 1024));
      }
    }
  }

  // load the next stage; after a tile's last one, next() seeks another tile or leaves `more` false
  template <bool TA, bool TB, class Next>
  __device__ __forceinline__ void load(Next&& next) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint8_t* const dst = lds + buf_load * STAGE;
    const int left = at_k < nfull ? KS : static_cast<int>(k1 - k0) - at_k * KS;
    load_operand<TA, BM, NLA>(ab, offa, dst + wave * NLA * 1024, wave, left);
    load_operand<TB, BN, NLB>(bb, offb, dst + ABYTES + wave * NLB * 1024, wave, left);
    buf_load = buf_load + 1 == NST ? 0 : buf_load + 1;
    ++ahead;
    ab += TA ? 2 * KS * A.ld : 2 * BK;
    bb += TB ? 2 * KS * B.ld : 2 * BK;
    if (++at_k == nk) {
      more = false;
      next();
    }
  }

  // the first stages of the first tile (after seek)
  template <bool TA, bool TB, class Next>
  __device__ __forceinline__ void prime(Next&& next) {
#pragma unroll
    for (int s = 0; s < NST - 1; ++s)
      if (more) load<TA, TB>(next);
  }

  // fragment of 32 tile rows from row `at`, k = 16 kb .., of a stage's rows / cols
  static __device__ __forceinline__ mm_bf16x8 frag_rows(const uint8_t* st, int at, int kb) {
    const int lane = threadIdx.x & 63, r = at + (lane & 31);
    return *reinterpret_cast<const mm_bf16x8*>(st + r * (2 * BK) + 16 * row_pos(r, 2 * kb + (lane >> 5)));
  }
  template <int ROWBYTES>
  static __device__ __forceinline__ mm_bf16x8 frag_cols(const uint8_t* st, int at, int kb) {
    const int lane = threadIdx.x & 63, grp = lane >> 4, jl = lane & 15;
    const int col = at + 16 * (grp & 1) + 4 * (jl & 3);
    mm_s16x8 v;
#pragma unroll
    for (int call = 0; call < 2; ++call) {
      const int k = 16 * kb + 8 * (grp >> 1) + (jl >> 2) + 4 * call;
      const uint8_t* a = st + k * ROWBYTES + 16 * ((col >> 3) ^ swz<ROWBYTES / 16>(k)) + 2 * (col & 7);
      const mm_s16x4 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) mm_s16x4*)(a));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * call + e] = r[e];
    }
    return __builtin_bit_cast(mm_bf16x8, v);
  }

  // acc = (or, with ADD, +=) the next tile's product (acc is left alone if the
  // summed range is empty).  `stored`: this wave has issued STORES stores, no
  // fewer, since the last stage was loaded; they may stay in flight (the
  // counter goes down in the order of issue).
  template <bool TA, bool TB, bool ADD = false, bool F16 = false, int STORES = 0, class Next>
  __device__ __forceinline__ void multiply(Next&& next, bool stored = false) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wr = wave / WC, wc = wave % WC;
    constexpr int KB = BK / 16;
    static_assert(KB % 2 == 0, "two sets of fragments in turn");
    const int stages = nk;
    if (stages == 0) return;
    const uint8_t* sa;
    // the next stage has landed, and every wave is done with the buffer that
    // the load after it fills
    auto arrive = [&](bool after_stores) {
      asm volatile("" ::: "memory");
      if (STORES && after_stores)
        mm_wait_loads<STORES>();
      else if (ahead >= NST - 1)
        mm_wait_loads<(NST - 2) * (NLA + NLB)>();
      else
        mm_wait_loads<0>();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (more) load<TA, TB>(next);
      --ahead;
      sa = lds + buf_use * STAGE;
      buf_use = buf_use + 1 == NST ? 0 : buf_use + 1;
    };
    mm_bf16x8 av[2][WM], bv[2][WN];
    auto fragments_a = [&](int kb, mm_bf16x8 (&a)[WM]) {
#pragma unroll
      for (int i = 0; i < WM; ++i) {
        const int at = (wr * WM + i) * 32;
        if constexpr (TA) a[i] = frag_cols<2 * BM>(sa, at, kb); else a[i] = frag_rows(sa, at, kb);
      }
    };
    auto fragments_b = [&](int kb, mm_bf16x8 (&b)[WN]) {
      const uint8_t* sb = sa + ABYTES;
#pragma unroll
      for (int j = 0; j < WN; ++j) {
        const int at = (wc * WN + j) * 32;
        if constexpr (TB) b[j] = frag_cols<2 * BN>(sb, at, kb); else b[j] = frag_rows(sb, at, kb);
      }
    };
    constexpr int kReadsA = WM * (TA ? 2 : 1), kReadsB = WN * (TB ? 2 : 1);
    // every product with a share of the next fragments behind it (left to
    // itself the compiler reads each fragment just before its use)
    auto in_order = [&](auto n) {
      constexpr int kReads = decltype(n)::value, kProducts = WM * WN, kMost = (kReads + kProducts - 1) / kProducts;
#pragma unroll
      for (int m = 0; m < kProducts; ++m) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        if (kReads > 0 && (m + 1) * kReads / kProducts > m * kReads / kProducts)
          __builtin_amdgcn_sched_group_barrier(0x100, kMost, 0);
      }
    };
    using None = std::integral_constant<int, 0>;
    using OfA = std::integral_constant<int, kReadsA>;
    using OfB = std::integral_constant<int, kReadsB>;
    using Both = std::integral_constant<int, kReadsA + kReadsB>;
    auto products = [&](int sa_, int sb_) {
#pragma unroll
      for (int i = 0; i < WM; ++i)
#pragma unroll
        for (int j = 0; j < WN; ++j) acc[i][j] = mm_product<F16>(av[sa_][i], bv[sb_][j], acc[i][j]);
    };
    auto first_products = [&](bool first) {
      if (first) {   // a tile's first products start from zero (cheaper than clearing acc)
        const mm_f32x16 zero = {};
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
          for (int j = 0; j < WN; ++j) acc[i][j] = mm_product<F16>(av[0][i], bv[0][j], zero);
      } else {
        products(0, 0);
      }
    };
    auto next_stage = [&]() {
      __builtin_amdgcn_sched_barrier(0);
      arrive(false);
      fragments_a(0, av[0]);
      fragments_b(0, bv[0]);
    };
    // a stage whose first fragments are in sets 0; but after the last one, the
    // next stage's are on their way there while the last products run.  The
    // last one stops at its blocks of 16 k (the rest are zeros).
    auto stage = [&](bool first, auto last) {
      constexpr bool LAST = decltype(last)::value;
      if constexpr (PAIR) {
        fragments_b(2, bv[1]);
        first_products(first);   // high high, k 0 .. 15
        fragments_a(2, av[1]);
        products(0, 1);          // high low
        in_order(OfA{});
        const bool more_k = !LAST || ntail > 1;
        if (more_k) {
          fragments_a(1, av[0]);
          fragments_b(1, bv[1]);
        }
        products(1, 0);          // low high
        if (!LAST) in_order(Both{});
        if (more_k) {            // k 16 .. 31
          fragments_b(3, bv[0]);
          products(0, 1);
          in_order(OfB{});
          fragments_a(3, av[1]);
          products(0, 0);
          in_order(OfA{});
          if constexpr (!LAST) next_stage();
          products(1, 1);
          in_order(std::conditional_t<LAST, None, Both>{});
        }
      } else {
        fragments_a(1, av[1]);
        fragments_b(1, bv[1]);
        first_products(first);
#pragma unroll
        for (int kb = 1; kb < KB; ++kb) {
          if (LAST && kb >= ntail) break;
          if (kb + 1 < KB) {
            fragments_a(kb + 1, av[(kb + 1) & 1]);
            fragments_b(kb + 1, bv[(kb + 1) & 1]);
          } else if constexpr (!LAST) {
            next_stage();
          }
          products(kb & 1, kb & 1);
          if (kb + 1 < KB || !LAST) in_order(Both{}); else in_order(None{});
        }
      }
    };
    arrive(stored);
    fragments_a(0, av[0]);
    fragments_b(0, bv[0]);
    for (int st = 0; st + 1 < stages; ++st) stage(!ADD && st == 0, std::false_type{});
    stage(!ADD && stages == 1, std::true_type{});
    __builtin_amdgcn_sched_barrier(0);   // an epilogue begins after the products: mixed with them it spills
  }
};

}  // namespace prn
