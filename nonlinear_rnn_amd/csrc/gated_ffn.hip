// Gated feed-forward product, and the gradients of its sums.
//
//   g = x Wg^T    u = x Wu^T    out = act(g) u        W = [Wg; Wu], 2 F x d
//   dg = dout u act'(g)         du = dout act(g)      (dx = [dg | du] W, dW = [dg | du]^T x)
//
// One kernel has both products: a tile's columns are pairs of a gate and an up
// row of W, so that the two sums of a pair meet in one lane's accumulators,
// in fp32, and only the result is stored.  The backward pass forms the sums
// again (4 N F d operations) instead of reading 2 N F stored values.
#include "gated_ffn.h"

#include <algorithm>

#include "grid_rows.h"
#include "proj.h"

namespace prn {
namespace {

size_t up(size_t x) { return (x + 255) / 256 * 256; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A copy of rows of d values as rows of ldp, zeros past d; a thread per 16 bytes.
template <class T>
__global__ void __launch_bounds__(256) k_ffn_pad(const T* __restrict__ in, int64_t R, int64_t d, int64_t ldp,
                                                 T* __restrict__ out) {
  constexpr int V = 16 / sizeof(T);
  const int64_t C = ldp / V, i = block_in_rows() * 256 + threadIdx.x;
  if (i >= R * C) return;
  const int64_t r = i / C, c0 = (i - r * C) * V;
  T v[V];
  if (c0 + V <= d) {
    __builtin_memcpy(v, in + r * d + c0, sizeof(v));   // aligned or not
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = c0 + e < d ? in[r * d + c0 + e] : T(0);
  }
  __builtin_memcpy(__builtin_assume_aligned(out + r * ldp + c0, 16), v, sizeof(v));
}

// rows of d that are no multiple of 16 bytes are laid out anew
struct Plan {
  bool pad;
  int64_t ldp;
  size_t x_off, w_off, end;
};
Plan plan_of(const GatedFfnArgs& a) {
  Plan p{};
  const int64_t vec = a.bf16 ? 8 : 4, elt = a.bf16 ? 2 : 4;
  p.pad = a.d % vec != 0;
  p.ldp = cdiv(a.d, vec) * vec;
  if (p.pad) {
    p.w_off = up(size_t(a.N) * p.ldp * elt);
    p.end = p.w_off + up(size_t(2 * a.F) * p.ldp * elt);
  }
  return p;
}

void product(const GatedFfnArgs& a, const Plan& p, const void* x, const void* W, const void* dout, void* out) {
  auto padded = [&](const void* in, int64_t R, size_t off) {
    void* const to = a.ws + off;
    const dim3 grid = rows_of_blocks(cdiv(R * (p.ldp / (a.bf16 ? 8 : 4)), 256));
    if (a.bf16)
      k_ffn_pad<uint16_t><<<grid, 256, 0, a.stream>>>(static_cast<const uint16_t*>(in), R, a.d, p.ldp, static_cast<uint16_t*>(to));
    else
      k_ffn_pad<float><<<grid, 256, 0, a.stream>>>(static_cast<const float*>(in), R, a.d, p.ldp, static_cast<float*>(to));
    return to;
  };
  if (p.pad) {
    x = padded(x, a.N, p.x_off);
    W = padded(W, 2 * a.F, p.w_off);
  }
  launch_proj_gated(a.bf16, x, W, out, a.N, p.ldp, GatedProj{dout, a.F, a.silu}, a.stream);
}

}  // namespace

bool gated_ffn_fits(const GatedFfnArgs& a) {
  // tiles of 128 x 128, 256 threads each, below 2^32 threads
  return double(cdiv(a.N, 128)) * double(cdiv(a.F, 64)) < double(1 << 24) && 2.0 * double(a.F) * double(a.d) < 4294967296.0;
}

size_t gated_ffn_workspace(const GatedFfnArgs& a) { return a.N ? plan_of(a).end : 0; }

void launch_gated_ffn(const GatedFfnArgs& a, const void* x, const void* W, void* out) {
  product(a, plan_of(a), x, W, nullptr, out);
}

size_t gated_ffn_dz_workspace(const GatedFfnArgs& a, size_t* dz_at) {
  const Plan p = plan_of(a);
  *dz_at = p.end;
  return p.end + up(size_t(a.N) * 2 * a.F * (a.bf16 ? 2 : 4));
}

void launch_gated_ffn_dz(const GatedFfnArgs& a, const void* x, const void* W, const void* dout) {
  const Plan p = plan_of(a);
  product(a, p, x, W, dout, a.ws + p.end);
}

}  // namespace prn
