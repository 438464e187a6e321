"""Float64 reference of the linear-recurrence block: the gated linear
recurrence, one step after another, the gated feed-forward product and
dropout, with their gradients from the formulas, and the sizes that error
bounds are made of."""
from __future__ import annotations

import numpy as np


def sig(x):
    """The logistic function, without overflow."""
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def _segments(B, T, cu):
    """(row, first step, past the last step) of every sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(lo), int(hi)) for lo, hi in zip(cu[:-1], cu[1:])]


def _parts(cell, x):
    f, g = sig(x[:, :, 0]), sig(-x[:, :, 0])
    if cell == "glr":
        return f, g, g, f, x[:, :, 1]
    return f, g, sig(x[:, :, 1]), sig(-x[:, :, 1]), x[:, :, 2]


def gated_scan(cell, x, h0=None, cu=None):
    """x (B, T, G, d) -> states (B, T, d), final states (rows, 1, d)."""
    B, T, _, d = x.shape
    f, _, i, _, v = _parts(cell, x)
    segs = _segments(B, T, cu)
    H, last = np.zeros((B, T, d)), np.zeros((len(segs), 1, d))
    for j, (b, lo, hi) in enumerate(segs):
        h = np.zeros(d) if h0 is None else h0[j, 0]
        for t in range(lo, hi):
            h = f[b, t] * h + i[b, t] * v[b, t]
            H[b, t] = h
        last[j, 0] = h
    return H, last


def gated_scan_backward(cell, x, dH, h0=None, cu=None, dlast=None):
    """dxproj (B, T, G, d) and dh0 (rows, 1, d)."""
    B, T, G, d = x.shape
    f, nf, i, ni, v = _parts(cell, x)
    H, _ = gated_scan(cell, x, h0, cu)
    segs = _segments(B, T, cu)
    dx, dh0 = np.zeros(x.shape), np.zeros((len(segs), 1, d))
    for j, (b, lo, hi) in enumerate(segs):
        m = np.zeros(d) if dlast is None else dlast[j, 0].copy()
        for t in range(hi - 1, lo - 1, -1):
            lam = dH[b, t] + m
            prev = H[b, t - 1] if t > lo else (np.zeros(d) if h0 is None else h0[j, 0])
            dx[b, t, 0] = lam * (prev - v[b, t] if cell == "glr" else prev) * f[b, t] * nf[b, t]
            if cell == "glri":
                dx[b, t, 1] = lam * v[b, t] * i[b, t] * ni[b, t]
            dx[b, t, G - 1] = lam * i[b, t]
            m = f[b, t] * lam
        dh0[j, 0] = m
    return dx, dh0


def gated_scan_bounds(cell, x, h0=None, cu=None, dH=None, dlast=None, start=0.0):
    """Bounds of what fp32 arithmetic may do to each output, in units of 2^-24, before the output's own rounding.

    A gate s(x) from 2^(-x log2 e): the exponent is off by |x| and its power and quotient by 4 more, so a gate is off
    by k = |x| + 4 of itself; a step's product and sum add 2, a map's product 1: k + 3 for f h, k + 4 for i v.  What a
    step leaves is carried by the gates after it.  start: the relative error of stored states that the gradient
    begins its chunks from, in the same units."""
    B, T, G, d = x.shape
    f, nf, i, ni, v = _parts(cell, x)
    kf = np.abs(x[:, :, 0]) + 8
    ki = (np.abs(x[:, :, 1]) if cell == "glri" else np.abs(x[:, :, 0])) + 8
    av = np.abs(v)
    segs = _segments(B, T, cu)
    out = {"H": np.zeros((B, T, d)), "last": np.zeros((len(segs), 1, d))}
    size, before, bound_before = np.zeros((B, T, d)), np.zeros((B, T, d)), np.zeros((B, T, d))
    for j, (b, lo, hi) in enumerate(segs):
        s = np.zeros(d) if h0 is None else np.abs(h0[j, 0])
        e = np.zeros(d)
        for t in range(lo, hi):
            before[b, t], bound_before[b, t] = s, e
            e = f[b, t] * (e + kf[b, t] * s) + ki[b, t] * i[b, t] * av[b, t]
            s = f[b, t] * s + i[b, t] * av[b, t]
            out["H"][b, t], size[b, t] = e, s
        out["last"][j, 0] = e
    if dH is None:
        return out
    dx, dh0 = np.zeros(x.shape), np.zeros((len(segs), 1, d))
    for j, (b, lo, hi) in enumerate(segs):
        s = np.zeros(d) if dlast is None else np.abs(dlast[j, 0])
        e = np.zeros(d)
        for t in range(hi - 1, lo - 1, -1):
            ls, le = np.abs(dH[b, t]) + s, e + np.abs(dH[b, t]) + s
            p = before[b, t] + (av[b, t] if cell == "glr" else 0.0)
            pe = bound_before[b, t] + start * before[b, t] + p
            df = f[b, t] * nf[b, t]
            dx[b, t, 0] = df * (le * p + ls * pe + ls * p * (2 * kf[b, t] + 4))
            if cell == "glri":
                dx[b, t, 1] = i[b, t] * ni[b, t] * av[b, t] * (le + ls * (2 * ki[b, t] + 4))
            dx[b, t, G - 1] = i[b, t] * (le + ls * (ki[b, t] + 2))
            e = f[b, t] * (le + kf[b, t] * ls)
            s = f[b, t] * ls
        dh0[j, 0] = e
    return {**out, "dxproj": dx, "dh0": dh0}


def act(kind, g):
    return g * sig(g) if kind == "silu" else sig(g)


def slope(kind, g):
    return sig(g) * (1.0 + g * sig(-g)) if kind == "silu" else sig(g) * sig(-g)


def gated_ffn(x, W, kind="silu"):
    g, u = np.split(x @ W.T, 2, axis=-1)
    return act(kind, g) * u


def gated_ffn_backward(x, W, dout, kind="silu"):
    g, u = np.split(x @ W.T, 2, axis=-1)
    dz = np.concatenate([dout * u * slope(kind, g), dout * act(kind, g)], -1)
    return dz @ W, dz.T @ x


def gated_ffn_bounds(x, W, kind, dout=None, rounding=0.0):
    """Bounds of out, dx and dW before their own rounding; rounding: that of the stored gradients of the sums,
    relative.  A sum of n products is off by (n + 8) 2^-24 of the sum of their magnitudes (each product's terms that
    are left out are within 3 of the 8)."""
    u24 = 2.0 ** -24
    d, F = x.shape[1], W.shape[0] // 2
    g, u = np.split(x @ W.T, 2, axis=-1)
    eg, eu = np.split((d + 8) * u24 * (np.abs(x) @ np.abs(W).T), 2, axis=-1)
    a, s = np.abs(act(kind, g)), np.abs(slope(kind, g))
    k = (np.abs(g) + 10) * u24             # the gate itself, as in gated_scan_bounds
    # |slope| <= 1.1, |slope'| <= 0.5 for both
    ea = 1.1 * eg + k * (np.abs(g) * sig(g) + a)
    es = 0.5 * eg + 2 * k * (1.0 + np.abs(g) * sig(-g)) * sig(g) + 2 * k * s
    out = ea * np.abs(u) + a * eu + ea * eu + 4 * u24 * a * np.abs(u)
    if dout is None:
        return out
    ad = np.abs(dout)
    dz = np.concatenate([ad * np.abs(u) * s, ad * a], -1)
    ez = np.concatenate([ad * (es * np.abs(u) + s * eu + es * eu), ad * ea], -1) + (4 * u24 + rounding) * dz
    ez *= 1.0 + rounding
    N = x.shape[0]
    return (out, ez @ np.abs(W) + (2 * F + 8) * u24 * ((dz + ez) @ np.abs(W)),
            ez.T @ np.abs(x) + (N + 8) * u24 * ((dz + ez).T @ np.abs(x)))


def philox(block, offset, seed):
    """Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011): four words for every 64-bit block number."""
    m = (1 << 32) - 1
    out = np.empty((len(block), 4), dtype=np.uint32)
    for n, b in enumerate(block):
        c = [int(b) & m, int(b) >> 32, offset & m, (offset >> 32) & m]
        k = [seed & m, (seed >> 32) & m]
        for _ in range(10):
            p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
            c = [(q >> 32) ^ c[1] ^ k[0], q & m, (p >> 32) ^ c[3] ^ k[1], p & m]
            k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
        out[n] = c
    return out


def kept(n, p, seed, offset):
    """Which of n elements stay."""
    words = philox(np.arange((n + 7) // 8), offset, seed)
    halves = np.stack([words & 0xFFFF, words >> 16], -1).reshape(-1)
    return halves[:n] >= round(p * 65536)


def dropout(x, p, seed, offset, residual=None):
    keep = kept(x.size, p, seed, offset).reshape(x.shape)
    q = round(p * 65536) / 65536
    y = np.where(keep, x / (1.0 - q) if q < 1.0 else 0.0, 0.0)
    return y if residual is None else residual + y
