"""The operators of a token model around the recurrence, plainly, in float64:
embedding lookup, the norms at a block boundary, and the softmax cross entropy
over a vocabulary, with their gradients.  Gradients are pinned by central
differences (tests/test_oracle_lm.py).

Functions named ``*_scale`` give, for every result, the same formula over
absolute values: the size that floating-point errors are measured against.
"""
from __future__ import annotations

import numpy as np


def embed(tokens, table, scale=1.0, pad_id=None):
    out = np.full((len(tokens), table.shape[1]), np.nan)
    for n, t in enumerate(tokens):
        if pad_id is not None and t == pad_id:
            out[n] = 0.0
        elif 0 <= t < table.shape[0]:
            out[n] = scale * table[t]
    return out


def embed_backward(dout, tokens, V, scale=1.0, pad_id=None):
    """(gradient, sums of |scale dout|, number of rows summed) per table row."""
    grad, size, count = np.zeros((V, dout.shape[1])), np.zeros((V, dout.shape[1])), np.zeros(V, dtype=np.int64)
    live = (tokens >= 0) & (tokens < V)
    if pad_id is not None:
        live &= tokens != pad_id
    np.add.at(grad, tokens[live], scale * dout[live])
    np.add.at(size, tokens[live], np.abs(scale * dout[live]))
    np.add.at(count, tokens[live], 1)
    return grad, size, count


def _act(g, act, size=False):
    """(act(g), act'(g)); size: over absolute values (silu' = s + g s (1 - s) changes sign near -1.28)."""
    s = 1.0 / (1.0 + np.exp(-g))
    g = np.abs(g) if size else g
    return (g * s, s * (1.0 + g * (1.0 - s))) if act == "silu" else (s, s * (1.0 - s))


def block_norm(h, x=None, gate=None, w_post=None, w_pre=None, alpha=None, act="silu", eps=1e-6):
    rstd = lambda y: 1.0 / np.sqrt((y * y).mean(-1, keepdims=True) + eps)   # noqa: E731
    u = h if w_post is None else h * rstd(h) * w_post
    v = u if gate is None else u * _act(gate, act)[0]
    r = v if alpha is None else alpha * v
    r = r if x is None else x + r
    return r, (None if w_pre is None else r * rstd(r) * w_pre)


def block_norm_backward(dr, dn, h, x=None, gate=None, w_post=None, w_pre=None, alpha=None, act="silu", eps=1e-6,
                        size=False):
    """dict of gradients.  size: every sum taken over absolute values instead (r as |x| + |alpha v|)."""
    a = np.abs if size else (lambda y: y)
    sub = 1.0 if size else -1.0
    mean = lambda y: y.mean(-1, keepdims=True)   # noqa: E731
    rstd_h = 1.0 / np.sqrt(mean(h * h) + eps) if w_post is not None else 1.0
    hn = a(h) * rstd_h
    wo = 1.0 if w_post is None else a(w_post)
    al = 1.0 if alpha is None else a(alpha)
    f, df = (1.0, None) if gate is None else _act(gate, act, size)
    v = hn * wo * f
    R = np.zeros_like(h) if dr is None else a(dr)
    out = {}
    if w_pre is not None:
        r_true = block_norm(h, x, gate, w_post, None, alpha, act, eps)[0]
        rstd_r = 1.0 / np.sqrt(mean(r_true * r_true) + eps)
        r = al * v if x is None else a(x) + al * v
        rn = r * rstd_r
        q = a(dn) * a(w_pre)
        out["dw_pre"] = (a(dn) * rn).sum(0)
        R = R + rstd_r * (q + sub * rn * mean(q * rn))
    if x is not None:
        out["dx"] = R
    if alpha is not None:
        out["dalpha"] = (R * v).sum(0)
    dv = R * al
    if gate is not None:
        out["dgate"] = dv * hn * wo * df
    du = dv * f
    if w_post is not None:
        out["dw_post"] = (du * hn).sum(0)
        p = du * wo
        du = rstd_h * (p + sub * hn * mean(p * hn))
    out["dh"] = du
    return out


def vocab_loss(x, W, targets, scale=1.0, ignore_index=-100):
    """(loss, lse, z)."""
    z = scale * (x @ W.T)
    m = z.max(-1, keepdims=True)
    lse = (np.log(np.exp(z - m).sum(-1, keepdims=True)) + m)[:, 0]
    loss = np.full(len(targets), np.nan)
    for n, t in enumerate(targets):
        if t == ignore_index:
            loss[n] = 0.0
        elif 0 <= t < W.shape[0]:
            loss[n] = lse[n] - z[n, t]
    return loss, lse, z


def vocab_loss_dz(dloss, dlse, z, lse, targets, scale=1.0, ignore_index=-100):
    """dL/d(x W^T): (N, V).  Rows of targets out of range are NaN."""
    V = z.shape[1]
    p = np.exp(z - lse[:, None])
    one = np.where(targets == ignore_index, 0.0, dloss)
    dz = p * (one if dlse is None else one + dlse)[:, None]
    for n, t in enumerate(targets):
        if t == ignore_index:
            continue
        if 0 <= t < V:
            dz[n, t] -= one[n]
        else:
            dz[n] = np.nan
    return scale * dz
