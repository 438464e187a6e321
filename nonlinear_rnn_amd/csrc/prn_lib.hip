// The library's host side: the recurrence's entry points (prn_api.hip) and
// those of the token model around it, in one translation unit, since they
// share the thread's error message and the argument helpers.
//
// Here: argument checks, workspace checks and launches of prn_embed*,
// prn_block_norm* and prn_vocab_loss*.
#include "prn_api.hip"

#include "block_norm.h"
#include "embed.h"
#include "vocab_loss.h"

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

prn_status check_dtype(int32_t dtype) {
  if (dtype != PRN_F32 && dtype != PRN_BF16) return fail(PRN_ERR_INVALID_ARG, "unknown storage dtype %d", dtype);
  return PRN_OK;
}
prn_status check_id_bytes(int32_t bytes, const char* what) {
  if (bytes != 4 && bytes != 8) return fail(PRN_ERR_INVALID_ARG, "%s must be 4 or 8, got %d", what, bytes);
  return PRN_OK;
}
prn_status check_scratch(const void* ws, size_t have, size_t need) {
  if (need && (!ws || have < need))
    return fail(PRN_ERR_WORKSPACE, "workspace of %zu bytes at %p; %zu bytes needed", have, ws, need);
  if (need && reinterpret_cast<uintptr_t>(ws) % kAlign)
    return fail(PRN_ERR_WORKSPACE, "workspace must be %zu-byte aligned", kAlign);
  return PRN_OK;
}
bool is_finite(float v) { return v - v == 0.0f; }

prn_status embed_args(const prn_embed_params* p, prn::EmbedArgs* a) {
  if (!p) return fail(PRN_ERR_INVALID_ARG, "params is NULL");
  if (prn_status s = check_dtype(p->dtype); s != PRN_OK) return s;
  if (prn_status s = check_id_bytes(p->token_bytes, "token_bytes"); s != PRN_OK) return s;
  if (p->N < 0 || p->V < 1 || p->d < 1)
    return fail(PRN_ERR_INVALID_ARG, "bad sizes N=%lld V=%lld d=%lld", (long long)p->N, (long long)p->V, (long long)p->d);
  if (p->N > kMaxRows || p->V >= kMaxRows || p->d > (int64_t(1) << 20))
    return fail(PRN_ERR_UNSUPPORTED, "N below 2^31, V below 2^31 - 1 and d up to 2^20; got N=%lld V=%lld d=%lld",
                (long long)p->N, (long long)p->V, (long long)p->d);
  *a = {p->dtype == PRN_BF16, p->token_bytes, p->N, p->V, p->d, p->scale, p->pad_id,
        static_cast<uint8_t*>(p->workspace), static_cast<hipStream_t>(p->stream)};
  return PRN_OK;
}

prn_status norm_args(const prn_block_norm_params* p, prn::BlockNormArgs* a) {
  if (!p) return fail(PRN_ERR_INVALID_ARG, "params is NULL");
  if (prn_status s = check_dtype(p->dtype); s != PRN_OK) return s;
  if (p->act != PRN_ACT_SILU && p->act != PRN_ACT_SIGMOID)
    return fail(PRN_ERR_INVALID_ARG, "unknown gate activation %d", p->act);
  if (p->N < 0 || p->d < 1) return fail(PRN_ERR_INVALID_ARG, "bad sizes N=%lld d=%lld", (long long)p->N, (long long)p->d);
  if (p->N > kMaxRows || p->d > prn::kBlockNormMaxWidth)
    return fail(PRN_ERR_UNSUPPORTED, "N below 2^31 and d up to %lld; got N=%lld d=%lld",
                (long long)prn::kBlockNormMaxWidth, (long long)p->N, (long long)p->d);
  if (!is_finite(p->eps) || p->eps < 0.0f) return fail(PRN_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (misaligned(p->w_post, 4) || misaligned(p->w_pre, 4) || misaligned(p->alpha, 4))
    return fail(PRN_ERR_INVALID_ARG, "a weight pointer is not 4-byte aligned");
  *a = prn::BlockNormArgs{};
  a->bf16 = p->dtype == PRN_BF16;
  a->act = p->act;
  a->N = p->N;
  a->d = p->d;
  a->eps = p->eps;
  a->w_post = p->w_post;
  a->w_pre = p->w_pre;
  a->alpha = p->alpha;
  a->ws = static_cast<uint8_t*>(p->workspace);
  a->stream = static_cast<hipStream_t>(p->stream);
  return PRN_OK;
}

prn_status loss_args(const prn_vocab_loss_params* p, prn::LossArgs* a) {
  if (!p) return fail(PRN_ERR_INVALID_ARG, "params is NULL");
  if (prn_status s = check_dtype(p->dtype); s != PRN_OK) return s;
  if (prn_status s = check_id_bytes(p->target_bytes, "target_bytes"); s != PRN_OK) return s;
  if (p->N < 0 || p->V < 1 || p->d < 1)
    return fail(PRN_ERR_INVALID_ARG, "bad sizes N=%lld V=%lld d=%lld", (long long)p->N, (long long)p->V, (long long)p->d);
  if (p->N > kMaxRows || p->V > (int64_t(1) << 31) - 1024 || p->d >= (int64_t(1) << 20))
    return fail(PRN_ERR_UNSUPPORTED, "N below 2^31, V up to 2^31 - 1024 and d below 2^20; got N=%lld V=%lld d=%lld",
                (long long)p->N, (long long)p->V, (long long)p->d);
  if (!is_finite(p->scale) || !(p->scale > 0.0f)) return fail(PRN_ERR_INVALID_ARG, "scale must be finite and > 0");
  *a = {p->dtype == PRN_BF16, p->target_bytes, p->N, p->V, p->d, p->scale, p->ignore_index,
        static_cast<uint8_t*>(p->workspace), static_cast<hipStream_t>(p->stream)};
  if (!prn::loss_fits(*a)) return fail(PRN_ERR_UNSUPPORTED, "too many tiles for one launch: N=%lld V=%lld",
                                       (long long)p->N, (long long)p->V);
  return PRN_OK;
}

}  // namespace

extern "C" {

prn_status prn_embed(const void* tokens, const void* table, const prn_embed_params* p, void* out) {
  prn::EmbedArgs a;
  if (prn_status s = embed_args(p, &a); s != PRN_OK) return s;
  if (!table) return fail(PRN_ERR_INVALID_ARG, "table is NULL");
  if (a.N && (!tokens || !out)) return fail(PRN_ERR_INVALID_ARG, "tokens or out is NULL");
  const size_t elt = a.bf16 ? 2 : 4;
  if (misaligned(table, elt) || misaligned(out, elt) || misaligned(tokens, a.token_bytes))
    return fail(PRN_ERR_INVALID_ARG, "a tensor pointer is not aligned to its element size");
  if (!a.N) return PRN_OK;
  prn::launch_embed(a, tokens, table, out);
  return launched("prn_embed");
}

size_t prn_embed_backward_workspace_bytes(const prn_embed_params* p) {
  g_err.clear();
  prn::EmbedArgs a;
  if (embed_args(p, &a) != PRN_OK) return 0;
  return prn::embed_backward_workspace(a);
}

prn_status prn_embed_backward(const void* tokens, const void* dout, const prn_embed_params* p, void* dtable) {
  prn::EmbedArgs a;
  if (prn_status s = embed_args(p, &a); s != PRN_OK) return s;
  if (!dtable) return fail(PRN_ERR_INVALID_ARG, "dtable_out is NULL");
  if (a.N && (!tokens || !dout)) return fail(PRN_ERR_INVALID_ARG, "tokens or dout is NULL");
  if (misaligned(dtable, 16)) return fail(PRN_ERR_INVALID_ARG, "dtable_out must be 16-byte aligned");
  if (misaligned(dout, a.bf16 ? 2 : 4) || misaligned(tokens, a.token_bytes))
    return fail(PRN_ERR_INVALID_ARG, "a tensor pointer is not aligned to its element size");
  if (prn_status s = check_scratch(p->workspace, p->workspace_bytes, prn::embed_backward_workspace(a)); s != PRN_OK)
    return s;
  prn::launch_embed_backward(a, tokens, dout, dtable);
  return launched("prn_embed_backward");
}

prn_status prn_block_norm(const void* h, const void* gate, const void* x, const prn_block_norm_params* p, void* r_out,
                          void* n_out) {
  prn::BlockNormArgs a;
  if (prn_status s = norm_args(p, &a); s != PRN_OK) return s;
  if (a.N && !h) return fail(PRN_ERR_INVALID_ARG, "h is NULL");
  if (a.N && (n_out != nullptr) != (a.w_pre != nullptr))
    return fail(PRN_ERR_INVALID_ARG, "n_out is given exactly when w_pre is");
  if (a.N && !r_out && !n_out) return fail(PRN_ERR_INVALID_ARG, "neither r_out nor n_out is given");
  if (misaligned(h, 16) || misaligned(gate, 16) || misaligned(x, 16) || misaligned(r_out, 16) || misaligned(n_out, 16))
    return fail(PRN_ERR_INVALID_ARG, "h, gate, x, r_out and n_out must be 16-byte aligned");
  if (!a.N) return PRN_OK;
  a.h = h, a.gate = gate, a.x = x, a.r_out = r_out, a.n_out = n_out;
  prn::launch_block_norm(a);
  return launched("prn_block_norm");
}

size_t prn_block_norm_backward_workspace_bytes(const prn_block_norm_params* p) {
  g_err.clear();
  prn::BlockNormArgs a;
  if (norm_args(p, &a) != PRN_OK) return 0;
  return prn::block_norm_backward_workspace(a.bf16, a.N, a.d);
}

prn_status prn_block_norm_backward(const void* h, const void* gate, const void* x, const void* dr, const void* dn,
                                   const prn_block_norm_params* p, void* dh, void* dgate, void* dx, float* dw_post,
                                   float* dw_pre, float* dalpha) {
  prn::BlockNormArgs a;
  if (prn_status s = norm_args(p, &a); s != PRN_OK) return s;
  if (a.N && !h) return fail(PRN_ERR_INVALID_ARG, "h is NULL");
  if (a.N && (dn != nullptr) != (a.w_pre != nullptr)) return fail(PRN_ERR_INVALID_ARG, "dn is given exactly when w_pre is");
  if ((dgate && a.N && !gate) || (dx && a.N && !x) || (dw_post && !a.w_post) || (dw_pre && !a.w_pre) || (dalpha && !a.alpha))
    return fail(PRN_ERR_INVALID_ARG, "a gradient is asked for whose input is absent");
  if (misaligned(h, 16) || misaligned(gate, 16) || misaligned(x, 16) || misaligned(dr, 16) || misaligned(dn, 16) ||
      misaligned(dh, 16) || misaligned(dgate, 16) || misaligned(dx, 16))
    return fail(PRN_ERR_INVALID_ARG, "the N x d tensors must be 16-byte aligned");
  if (misaligned(dw_post, 4) || misaligned(dw_pre, 4) || misaligned(dalpha, 4))
    return fail(PRN_ERR_INVALID_ARG, "a weight gradient is not 4-byte aligned");
  if (prn_status s = check_scratch(p->workspace, p->workspace_bytes, prn::block_norm_backward_workspace(a.bf16, a.N, a.d));
      s != PRN_OK)
    return s;
  a.h = h, a.gate = gate, a.x = x, a.dr = dr, a.dn = dn;
  a.dh = dh, a.dgate = dgate, a.dx = dx, a.dw_post = dw_post, a.dw_pre = dw_pre, a.dalpha = dalpha;
  prn::launch_block_norm_backward(a);
  return launched("prn_block_norm_backward");
}

size_t prn_vocab_loss_workspace_bytes(const prn_vocab_loss_params* p) {
  g_err.clear();
  prn::LossArgs a;
  if (loss_args(p, &a) != PRN_OK) return 0;
  return prn::loss_workspace(a);
}

size_t prn_vocab_loss_backward_workspace_bytes(const prn_vocab_loss_params* p) {
  g_err.clear();
  prn::LossArgs a;
  if (loss_args(p, &a) != PRN_OK) return 0;
  return prn::loss_backward_workspace(a);
}

prn_status prn_vocab_loss(const void* x, const void* W, const void* targets, const prn_vocab_loss_params* p,
                          float* loss, float* lse) {
  prn::LossArgs a;
  if (prn_status s = loss_args(p, &a); s != PRN_OK) return s;
  if (!W) return fail(PRN_ERR_INVALID_ARG, "W is NULL");
  if (a.N && (!x || !targets || !loss || !lse)) return fail(PRN_ERR_INVALID_ARG, "x, targets, loss_out or lse_out is NULL");
  if (misaligned(x, 16) || misaligned(W, 16)) return fail(PRN_ERR_INVALID_ARG, "x and W must be 16-byte aligned");
  if (misaligned(targets, a.target_bytes) || misaligned(loss, 4) || misaligned(lse, 4))
    return fail(PRN_ERR_INVALID_ARG, "a tensor pointer is not aligned to its element size");
  if (prn_status s = check_scratch(p->workspace, p->workspace_bytes, prn::loss_workspace(a)); s != PRN_OK) return s;
  if (!a.N) return PRN_OK;
  prn::launch_loss(a, x, W, targets, loss, lse);
  return launched("prn_vocab_loss");
}

prn_status prn_vocab_loss_backward(const void* x, const void* W, const void* targets, const float* lse,
                                   const float* dloss, const float* dlse, const prn_vocab_loss_params* p, void* dx,
                                   void* dW) {
  prn::LossArgs a;
  if (prn_status s = loss_args(p, &a); s != PRN_OK) return s;
  if (!W) return fail(PRN_ERR_INVALID_ARG, "W is NULL");
  if (a.N && (!x || !targets || !lse || !dloss)) return fail(PRN_ERR_INVALID_ARG, "x, targets, lse or dloss is NULL");
  if (misaligned(x, 16) || misaligned(W, 16) || misaligned(dx, 16) || misaligned(dW, 16))
    return fail(PRN_ERR_INVALID_ARG, "x, W, dx_out and dW_out must be 16-byte aligned");
  if (misaligned(targets, a.target_bytes) || misaligned(lse, 4) || misaligned(dloss, 4) || misaligned(dlse, 4))
    return fail(PRN_ERR_INVALID_ARG, "a tensor pointer is not aligned to its element size");
  if (prn_status s = check_scratch(p->workspace, p->workspace_bytes, prn::loss_backward_workspace(a)); s != PRN_OK)
    return s;
  if (!dx && !dW) return PRN_OK;
  prn::launch_loss_backward(a, x, W, targets, lse, dloss, dlse, dx, dW);
  return launched("prn_vocab_loss_backward");
}

}  // extern "C"
