"""A token model around the recurrence: the embedding lookup, the norms at a
block boundary with their gate and residual scale, the gated feed-forward
product, dropout, and the softmax cross entropy over a vocabulary, each with
its gradient.

As in ``api``: strided views (and views that do not start on 16 bytes) are
copied to a dense layout first, outputs and workspaces are allocated here, the
arithmetic is the library's.  Leading dimensions are rows: tokens of any
shape, activations (..., d).  The plain functions compute one direction; the
``*_apply`` functions are differentiable, once: a second derivative raises.
"""
from __future__ import annotations

import torch

from . import binding as B_
from .autograd import first as _first


def _rows(t):
    """t (..., d) as dense rows (N, d) that start on 16 bytes: itself where it is that already."""
    if t is None:
        return None
    if t.dim() != 2:
        t = t.reshape(-1, t.shape[-1])
    if not t.is_contiguous():
        t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _flat(t):
    """Ids or fp32 values of any shape as one dense row."""
    if t.dim() != 1:
        t = t.reshape(-1)
    return t if t.is_contiguous() else t.contiguous()


def _weight(t):
    if t is None:
        return None
    if t.dtype != torch.float32:
        t = t.to(torch.float32)
    return t if t.is_contiguous() else t.contiguous()


def _shaped(shape, **tensors):
    """Refuses a tensor of another shape: rows are flattened, so that one of as many rows in another order would
    be taken for the right one."""
    for name, t in tensors.items():
        if t is not None and t.shape != shape:
            raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


def _scratch(n: int, device) -> torch.Tensor:
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ embedding lookup ---

def embed(tokens, table, *, scale: float = 1.0, pad_id=None) -> torch.Tensor:
    """scale * table[tokens]: tokens (...) int32 or int64, table (V, d); (..., d).

    Tokens equal to pad_id give zeros; a token outside the table gives NaN."""
    ids = _flat(tokens)
    if not table.is_contiguous():
        table = table.contiguous()
    out = table.new_empty((ids.shape[0], table.shape[1]))
    B_.prn_embed(ids, table, out, scale=scale, pad_id=pad_id)
    return out if tokens.dim() == 1 else out.view(*tokens.shape, table.shape[1])


def embed_backward(dout, tokens, V: int, *, scale: float = 1.0, pad_id=None) -> torch.Tensor:
    """The table's gradient (V, d): scale * the sums of dout (..., d) over equal tokens, each in token order
    and fp32 (bitwise reproducible); rows of absent tokens are zeros."""
    ids = _flat(tokens)
    d = dout.shape[-1]
    _shaped((*tokens.shape, d), dout=dout)
    dout = dout.reshape(-1, d).contiguous()
    dtable = torch.empty((V, d), dtype=dout.dtype, device=dout.device)
    ws = _scratch(B_.prn_embed_backward_workspace_bytes(dout.dtype, ids.numel(), V, d), dout.device)
    B_.prn_embed_backward(ids, dout, dtable, scale=scale, pad_id=pad_id, workspace=ws)
    return dtable


class _EmbedFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, table, scale, pad_id):
        ctx.save_for_backward(tokens)
        ctx.V, ctx.scale, ctx.pad_id, ctx.dtype = table.shape[0], scale, pad_id, table.dtype
        return embed(tokens, table, scale=scale, pad_id=pad_id)

    @staticmethod
    def backward(ctx, dout):
        tokens, = ctx.saved_tensors
        dtable = embed_backward(dout.to(ctx.dtype), tokens, ctx.V, scale=ctx.scale, pad_id=ctx.pad_id)
        return None, *_first((dtable,), dout), None, None


def embed_apply(tokens, table, *, scale: float = 1.0, pad_id=None) -> torch.Tensor:
    """Differentiable embed."""
    return _EmbedFunction.apply(tokens, table, float(scale), pad_id)


# ------------------------------------------------------------------ block boundary ---

def block_norm(h, x=None, *, gate=None, w_post=None, w_pre=None, alpha=None, act: str = "silu", eps: float = 1e-6):
    """The boundary between two blocks, in one pass over the rows of h (..., d):

        u = h / rms(h) * w_post     r = x + alpha * u * act(gate)     n = r / rms(r) * w_pre

    with rms(y) = sqrt(mean(y^2) + eps) over the last dimension.  Returns (r, n).
    w_post, gate, x, alpha, w_pre may each be None (the step is then the
    identity, n is None without w_pre).  With w_pre alone r is h itself: the
    norm before the first block."""
    shape = h.shape
    _shaped(shape, x=x, gate=gate)
    h2, x2, g2 = _rows(h), _rows(x), _rows(gate)
    w_post, w_pre, alpha = _weight(w_post), _weight(w_pre), _weight(alpha)
    same = x2 is None and g2 is None and w_post is None and alpha is None
    if same and w_pre is None:
        raise ValueError("block_norm without any of its parts")
    r = h2 if same else torch.empty_like(h2)
    n = None if w_pre is None else torch.empty_like(h2)
    B_.prn_block_norm(h2, g2, x2, None if same else r, n, w_post=w_post, w_pre=w_pre, alpha=alpha, act=act, eps=eps)
    if len(shape) == 2:
        return (h if same else r), n
    return (h if same else r.view(shape)), (None if n is None else n.view(shape))


def block_norm_backward(dr, dn, h, x=None, *, gate=None, w_post=None, w_pre=None, alpha=None, act: str = "silu",
                        eps: float = 1e-6):
    """Gradients of block_norm from dr = dL/dr (None for zero) and dn = dL/dn (None without w_pre):
    (dh, dx, dgate, dw_post, dw_pre, dalpha), None where the input is absent; the weights' are fp32."""
    shape = h.shape
    _shaped(shape, x=x, gate=gate, dr=dr, dn=dn)
    h2, x2, g2, dr2, dn2 = _rows(h), _rows(x), _rows(gate), _rows(dr), _rows(dn)
    w_post, w_pre, alpha = _weight(w_post), _weight(w_pre), _weight(alpha)
    dh, dx, dgate = (None if t is None else torch.empty_like(h2) for t in (h2, x2, g2))
    dw_post, dw_pre, dalpha = (None if t is None else torch.empty_like(t) for t in (w_post, w_pre, alpha))
    ws = _scratch(B_.prn_block_norm_backward_workspace_bytes(h2.dtype, *h2.shape), h2.device)
    B_.prn_block_norm_backward(h2, g2, x2, dr2, dn2, w_post=w_post, w_pre=w_pre, alpha=alpha, act=act, eps=eps,
                               dh_out=dh, dgate_out=dgate, dx_out=dx, dw_post_out=dw_post, dw_pre_out=dw_pre,
                               dalpha_out=dalpha, workspace=ws)
    return (dh.view(shape), None if dx is None else dx.view(shape), None if dgate is None else dgate.view(shape),
            dw_post, dw_pre, dalpha)


class _BlockNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, x, gate, w_post, w_pre, alpha, act, eps):
        ctx.save_for_backward(h, x, gate, w_post, w_pre, alpha)
        ctx.act, ctx.eps = act, eps
        ctx.set_materialize_grads(False)
        r, n = block_norm(h, x, gate=gate, w_post=w_post, w_pre=w_pre, alpha=alpha, act=act, eps=eps)
        return (None if r is h else r), n   # the stream itself is not an output

    @staticmethod
    def backward(ctx, dr, dn):
        h, x, gate, w_post, w_pre, alpha = ctx.saved_tensors
        if w_pre is not None and dn is None:
            dn = torch.zeros_like(h)
        dr, dn = (None if t is None else t.to(h.dtype) for t in (dr, dn))
        dh, dx, dgate, dw_post, dw_pre, dalpha = _first(
            block_norm_backward(dr, dn, h, x, gate=gate, w_post=w_post, w_pre=w_pre, alpha=alpha, act=ctx.act,
                                eps=ctx.eps), dr, dn, h, x, gate, w_post, w_pre, alpha)
        return dh, dx, dgate, dw_post, dw_pre, dalpha, None, None


def block_norm_apply(h, x=None, *, gate=None, w_post=None, w_pre=None, alpha=None, act: str = "silu",
                     eps: float = 1e-6):
    """Differentiable block_norm: gradients reach h, x, gate, w_post, w_pre and alpha.  Nothing but the inputs is
    kept between the passes."""
    if x is None and gate is None and w_post is None and alpha is None and w_pre is not None:
        return h, _BlockNormFunction.apply(h, None, None, None, _weight(w_pre), None, act, float(eps))[1]
    return _BlockNormFunction.apply(h, x, gate, _weight(w_post), _weight(w_pre), _weight(alpha), act, float(eps))


# ------------------------------------------------------------------ loss ---

def vocab_loss(x, W, targets, *, scale: float = 1.0, ignore_index: int = -100):
    """Softmax cross entropy of the logits scale * x W^T over a vocabulary, without the logits in memory:
    x (..., d), W (V, d), targets (...) int32 or int64.  Returns (loss, lse), fp32, shaped like targets; loss is 0
    where targets == ignore_index and NaN where a target is out of range; lse is the log of the summed
    exponentials (-loss is the target's log probability)."""
    _shaped(x.shape[:-1], targets=targets)
    if W.dim() != 2:
        raise ValueError(f"W must have 2 dimensions, got {tuple(W.shape)}")
    x2, W, ids = _rows(x), _rows(W), _flat(targets)
    loss = torch.empty(x2.shape[0], dtype=torch.float32, device=x2.device)
    lse = torch.empty_like(loss)
    ws = _scratch(B_.prn_vocab_loss_workspace_bytes(x2.dtype, x2.shape[0], *W.shape), x2.device)
    B_.prn_vocab_loss(x2, W, ids, loss, lse, scale=scale, ignore_index=ignore_index, workspace=ws)
    return (loss, lse) if targets.dim() == 1 else (loss.view(targets.shape), lse.view(targets.shape))


def vocab_loss_backward(dloss, x, W, targets, lse, *, dlse=None, scale: float = 1.0, ignore_index: int = -100,
                        want_x: bool = True, want_W: bool = True):
    """Gradients (dx, dW) of vocab_loss from dloss and dlse (None for zero), both shaped like targets; each only if
    wanted, else None.  The logits are formed again, a piece of the vocabulary at a time."""
    _shaped(x.shape[:-1], targets=targets, lse=lse, dloss=dloss, dlse=dlse)
    if W.dim() != 2:
        raise ValueError(f"W must have 2 dimensions, got {tuple(W.shape)}")
    x2, W, ids = _rows(x), _rows(W), _flat(targets)
    dloss, lse = _flat(_weight(dloss)), _flat(_weight(lse))
    dlse = None if dlse is None else _flat(_weight(dlse))
    dx = torch.empty_like(x2) if want_x else None
    dW = torch.empty_like(W) if want_W else None
    ws = _scratch(B_.prn_vocab_loss_backward_workspace_bytes(x2.dtype, x2.shape[0], *W.shape), x2.device)
    B_.prn_vocab_loss_backward(x2, W, ids, lse, dloss, dlse=dlse, scale=scale, ignore_index=ignore_index, dx_out=dx,
                               dW_out=dW, workspace=ws)
    return (None if dx is None else dx.view(x.shape)), dW


class _VocabLossFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, targets, scale, ignore_index):
        loss, lse = vocab_loss(x, W, targets, scale=scale, ignore_index=ignore_index)
        ctx.save_for_backward(x, W, targets, lse)
        ctx.scale, ctx.ignore_index = scale, ignore_index
        ctx.set_materialize_grads(False)
        return loss, lse

    @staticmethod
    def backward(ctx, dloss, dlse):
        x, W, targets, lse = ctx.saved_tensors
        if dloss is None:
            dloss = torch.zeros_like(lse)
        dx, dW = vocab_loss_backward(dloss, x, W, targets, lse, dlse=dlse, scale=ctx.scale,
                                     ignore_index=ctx.ignore_index, want_x=ctx.needs_input_grad[0],
                                     want_W=ctx.needs_input_grad[1])
        return *_first((dx, dW), dloss, dlse, x, W), None, None, None


def vocab_loss_apply(x, W, targets, *, scale: float = 1.0, ignore_index: int = -100):
    """Differentiable vocab_loss: gradients of loss and lse reach x and W."""
    return _VocabLossFunction.apply(x, W, targets, float(scale), int(ignore_index))


# ------------------------------------------------------------------ feed-forward ---

def _dense(t):
    """t as a dense tensor that starts on 16 bytes: itself where it is that already."""
    if not t.is_contiguous():
        t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def gated_ffn(x, W, *, act: str = "silu") -> torch.Tensor:
    """act(x Wg^T) * (x Wu^T) in one kernel: x (..., d), W (2 F, d) = [Wg; Wu]; (..., F).  act "silu" or "sigmoid"."""
    if W.dim() != 2 or W.shape[0] % 2 or W.shape[1] != x.shape[-1]:
        raise ValueError(f"W must be (2 F, {x.shape[-1]}), got {tuple(W.shape)}")
    x2, W = _rows(x), _dense(W)
    N, d, F = *x2.shape, W.shape[0] // 2
    out = x2.new_empty((N, F))
    n = B_.prn_gated_ffn_workspace_bytes(x2.dtype, N, d, F)
    B_.prn_gated_ffn(x2, W, out, act=act, workspace=_scratch(n, x2.device) if n else None)
    return out if x.dim() == 2 else out.view(*x.shape[:-1], F)


def gated_ffn_backward(dout, x, W, *, act: str = "silu", want_x: bool = True, want_W: bool = True):
    """Gradients (dx, dW) of gated_ffn from dout (..., F); each only if wanted, else None.  The sums are formed
    again: nothing but x and W is kept between the passes."""
    if W.dim() != 2 or W.shape[0] % 2 or W.shape[1] != x.shape[-1]:
        raise ValueError(f"W must be (2 F, {x.shape[-1]}), got {tuple(W.shape)}")
    F = W.shape[0] // 2
    _shaped((*x.shape[:-1], F), dout=dout)
    x2, W, dout2 = _rows(x), _dense(W), _rows(dout)
    dx = torch.empty_like(x2) if want_x else None
    dW = torch.empty_like(W) if want_W else None
    ws = _scratch(B_.prn_gated_ffn_backward_workspace_bytes(x2.dtype, *x2.shape, F), x2.device)
    B_.prn_gated_ffn_backward(x2, W, dout2, act=act, dx_out=dx, dW_out=dW, workspace=ws)
    return (None if dx is None else dx.view(x.shape)), dW


class _GatedFfnFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, act):
        ctx.save_for_backward(x, W)
        ctx.act = act
        return gated_ffn(x, W, act=act)

    @staticmethod
    def backward(ctx, dout):
        x, W = ctx.saved_tensors
        dx, dW = gated_ffn_backward(dout.to(x.dtype), x, W, act=ctx.act, want_x=ctx.needs_input_grad[0],
                                    want_W=ctx.needs_input_grad[1])
        return *_first((dx, dW), dout, x, W), None


def gated_ffn_apply(x, W, *, act: str = "silu") -> torch.Tensor:
    """Differentiable gated_ffn."""
    return _GatedFfnFunction.apply(x, W, act)


# ------------------------------------------------------------------ dropout ---

def dropout(x, p: float, *, seed, offset: int = 0, residual=None) -> torch.Tensor:
    """residual + x / (1 - q) where x stays and residual (or 0) where it is dropped, a share q = p rounded to 2^-16
    of the elements.  Which ones is a function of (seed, offset, the element's index) alone: another offset for
    every use of a seed.  seed may be an int64 tensor (seed, offset) on the device, read when the kernel runs, so
    that a captured graph draws anew after it is changed."""
    _shaped(x.shape, residual=residual)
    x2 = _dense(x)
    r2 = None if residual is None else _dense(residual)
    out = torch.empty_like(x2)
    if isinstance(seed, torch.Tensor):
        if offset:
            raise ValueError("a seed on the device holds its offset itself")
        B_.prn_dropout(x2, out, p=p, state=seed, residual=r2)
    else:
        B_.prn_dropout(x2, out, p=p, seed=seed, offset=offset, residual=r2)
    return out


def dropout_backward(dout, p: float, *, seed, offset: int = 0) -> torch.Tensor:
    """The gradient of dropout at x, from the gradient dout at its result (residual's is dout itself): dout / (1 - q)
    where x stayed, zero where it was dropped, by the same seed and offset."""
    return dropout(dout, p, seed=seed, offset=offset)


class _DropoutFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset):
        state = isinstance(seed, torch.Tensor)
        if state:   # the backward's numbers are this call's, whatever the tensor holds by then
            seed = seed.clone()
        ctx.save_for_backward(*((seed,) if state else ()))
        ctx.args = (p, None if state else seed, offset)
        ctx.dtype, ctx.kept = x.dtype, residual is not None
        return dropout(x, p, seed=seed, offset=offset, residual=residual)

    @staticmethod
    def backward(ctx, dout):
        p, seed, offset = ctx.args
        if ctx.saved_tensors:
            seed, = ctx.saved_tensors
        dout = dout.to(ctx.dtype)
        dx = None
        if ctx.needs_input_grad[0]:
            dx, = _first((dropout_backward(dout, p, seed=seed, offset=offset),), dout)
        return dx, dout if ctx.kept else None, None, None, None


def dropout_apply(x, p: float, *, seed, offset: int = 0, residual=None) -> torch.Tensor:
    """Differentiable dropout: the mask is drawn again in the backward pass, nothing is kept but the seed."""
    return _DropoutFunction.apply(x, residual, float(p), seed, int(offset))
