"""GPU parity of the block boundary (norm, gate, residual scale, norm) and its
gradients against oracle.lm.

Bands, per element: u |ref| for the rounding to storage (u = torch.finfo.eps /
2), plus k 2^-24 times the same formula over absolute values.  k counts the
fp32 roundings in a result's longest chain: a row sum takes at most 8 additions
in a lane, 6 across the wave and 16 across waves, its mean and reciprocal root
4 more (one of them of a step and a half); the backward chains three such sums
and about 30 products; the gate's exponent adds |g| roundings of its own size:
k = 160 + 8 max|g|.  Sums over N rows take at most N more additions.  A shut
gate (sig(g) below fp32's 2^-126) reads as zero: 2^-110 absolute, that limit
times factors of up to 2^16.
"""
import itertools

import numpy as np
import pytest
import torch

import nonlinear_rnn_amd as prn
from gpu_helpers import TORCH_DT, say, to_f64
from nonlinear_rnn_amd import binding as B
from oracle import lm as olm

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24


def _inputs(N, d, dtype, parts, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = lambda on, s=1.0: (s * torch.randn(N, d, generator=g, device="cuda")).to(TORCH_DT[dtype]) if on else None   # noqa: E731
    weights = lambda on: torch.randn(d, generator=g, device="cuda") if on else None   # noqa: E731
    gate, post, pre, alpha, res = parts
    kw = dict(h=rows(True), x=rows(res, 2.0), gate=rows(gate), w_post=weights(post), w_pre=weights(pre),
              alpha=weights(alpha))
    return kw, rows(True), rows(pre)


def _np(kw):
    return {k: None if v is None else to_f64(v) for k, v in kw.items()}


def _check(N, d, dtype, parts, act="silu", eps=1e-6, seed=0, kw=None):
    say(f"[case] block norm N={N} d={d} {dtype} gate,post,pre,alpha,res={parts} {act}")
    kw, dr, dn = _inputs(N, d, dtype, parts, seed) if kw is None else kw
    u = torch.finfo(TORCH_DT[dtype]).eps / 2
    ref_in = _np(kw)
    k = 160 + (8 * float(np.abs(ref_in["gate"]).max()) if kw["gate"] is not None and N else 0)
    h, x = kw.pop("h"), kw.pop("x")
    r, n = prn.block_norm(h, x, **kw, act=act, eps=eps)
    rr, rn = olm.block_norm(**ref_in, act=act, eps=eps)
    al = 1.0 if ref_in["alpha"] is None else ref_in["alpha"]
    v = olm.block_norm(**{**ref_in, "x": None, "alpha": None, "w_pre": None}, act=act, eps=eps)[0]
    r_size = np.abs(al * v) + (0.0 if ref_in["x"] is None else np.abs(ref_in["x"]))
    assert (np.abs(to_f64(r) - rr) <= u * np.abs(rr) + k * E24 * r_size).all()
    if n is not None:
        rstd = 1.0 / np.sqrt((rr * rr).mean(-1, keepdims=True) + eps)
        size = r_size * rstd * np.abs(ref_in["w_pre"])
        assert (np.abs(to_f64(n) - rn) <= u * np.abs(rn) + k * E24 * (size + np.abs(rn) * (r_size * rstd).max(-1, keepdims=True))).all()
    got = dict(zip(("dh", "dx", "dgate", "dw_post", "dw_pre", "dalpha"),
                   prn.block_norm_backward(dr, dn, h, x, **kw, act=act, eps=eps)))
    ref = olm.block_norm_backward(to_f64(dr), None if dn is None else to_f64(dn), **ref_in, act=act, eps=eps)
    size = olm.block_norm_backward(to_f64(dr), None if dn is None else to_f64(dn), **ref_in, act=act, eps=eps, size=True)
    for name, t in got.items():
        if name not in ref:
            assert t is None
            continue
        rows = name in ("dh", "dx", "dgate")
        band = ((u * np.abs(ref[name]) + k * E24 * size[name]) if rows else (k + N) * E24 * size[name]) + 2.0 ** -110
        err = np.abs(to_f64(t) - ref[name])
        worst = np.unravel_index((err / band).argmax(), err.shape)
        assert (err <= band).all(), (name, worst, float(err[worst]), float(band[worst]), float(ref[name][worst]))
    again = prn.block_norm_backward(dr, dn, h, x, **kw, act=act, eps=eps)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got.values(), again))


FULL = (True,) * 5


@pytest.mark.parametrize("parts", [p for p in itertools.product([False, True], repeat=5) if any(p)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_combination_of_parts(parts, dtype):
    _check(37, 72, dtype, parts, act="silu" if sum(parts) % 2 else "sigmoid", seed=sum(parts))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,d", [
    (1, 1), (5, 2), (3, 8), (300, 16), (33, 63), (65, 64), (9, 65), (2, 128), (70, 129), (129, 256), (5, 511), (64, 512),
    (66, 513), (7, 1001), (4, 1024), (3, 2048), (5, 2049), (2, 2056), (3, 4096), (2, 4100), (2, 4097), (3, 8191), (2, 8192),
    (5000, 24), (3000, 512)])
def test_widths_and_row_counts(N, d, dtype):
    _check(N, d, dtype, FULL, seed=N + d)
    _check(N, d, dtype, (False, False, True, False, False), seed=N + d + 1)


def test_rows_of_zeros_large_values_and_one_bad_row():
    kw, dr, dn = _inputs(6, 96, "f32", FULL, 3)
    kw["h"][1] = 0
    kw["x"][1] = 0
    kw["h"][2] *= 1e6
    kw["gate"][3] = -200.0      # a gate that is shut
    kw["gate"][4] = 50.0        # and one that is open
    _check(6, 96, "f32", FULL, kw=(dict(kw), dr, dn))
    # a row of NaN stays in its row (the weights' sums take it)
    bad = {k: v.clone() for k, v in kw.items()}
    bad["h"][0] = float("nan")
    good, gb = ({k: v for k, v in t.items() if k not in ("h", "x")} for t in (kw, bad))
    a, b = prn.block_norm(kw["h"], kw["x"], **good), prn.block_norm(bad["h"], bad["x"], **gb)
    for p, q in zip(a, b):
        assert q[0].isnan().all() and torch.equal(p[1:], q[1:])
    a = prn.block_norm_backward(dr, dn, kw["h"], kw["x"], **good)
    b = prn.block_norm_backward(dr, dn, bad["h"], bad["x"], **gb)
    for p, q in zip(a[:3], b[:3]):
        assert torch.equal(p[1:], q[1:])
    # eps = 0 and a row of zeros: 0 * inf, as the formula has it
    z = prn.block_norm(torch.zeros(2, 8, device="cuda"), w_pre=torch.ones(8, device="cuda"), eps=0.0)[1]
    assert z.isnan().all()


def test_empty_strided_misaligned_and_leading_dimensions():
    kw, dr, dn = _inputs(24, 40, "bf16", FULL, 5)
    h, x = kw.pop("h"), kw.pop("x")
    want = prn.block_norm(h, x, **kw)
    back = prn.block_norm_backward(dr, dn, h, x, **kw)
    got = prn.block_norm(h.view(2, 12, 40), x.view(2, 12, 40), **{**kw, "gate": kw["gate"].view(2, 12, 40)})
    assert all(g.shape == (2, 12, 40) and torch.equal(g.view(24, 40), w) for g, w in zip(got, want))
    wide = torch.zeros(24, 50, device="cuda", dtype=h.dtype)
    wide[:, 3:43] = h
    assert torch.equal(prn.block_norm(wide[:, 3:43], x, **kw)[1], want[1])
    flat = torch.empty(24 * 40 + 1, device="cuda", dtype=h.dtype)
    flat[1:] = h.view(-1)
    off = flat[1:].view(24, 40)
    assert torch.equal(prn.block_norm(off, x, **kw)[0], want[0])
    assert torch.equal(prn.block_norm_backward(dr, dn, off, x, **kw)[0], back[0])
    with pytest.raises(B.PrnError, match="16-byte"):
        B.prn_block_norm(off, None, None, h.clone(), None)
    e = h[:0]
    r, n = prn.block_norm(e, e, w_pre=kw["w_pre"])
    assert r.shape == n.shape == (0, 40)
    g = prn.block_norm_backward(e, e, e, e, w_pre=kw["w_pre"])
    assert g[0].shape == (0, 40) and not g[4].any()
    # a gradient that does not arrive along the stream
    none = prn.block_norm_backward(None, dn, h, x, **kw)
    zero = prn.block_norm_backward(torch.zeros_like(dr), dn, h, x, **kw)
    assert all(torch.equal(a, b) for a, b in zip(none, zero))


def test_in_place_outputs():
    kw, _, _ = _inputs(50, 520, "bf16", FULL, 6)
    h, x = kw.pop("h"), kw.pop("x")
    want = prn.block_norm(h, x, **kw)
    r, n, g = x.clone(), h.clone(), kw.pop("gate")
    B.prn_block_norm(n, g, r, r, n, **kw)
    assert torch.equal(r, want[0]) and torch.equal(n, want[1])


def test_autograd_against_differences():
    kw, dr, dn = _inputs(9, 20, "f32", FULL, 7)
    leaves = {k: v.clone().requires_grad_() for k, v in kw.items()}
    h, x = leaves["h"], leaves["x"]
    r, n = prn.block_norm_apply(h, x, **{k: v for k, v in leaves.items() if k not in ("h", "x")})
    ((r * dr).sum() + (n * dn).sum()).backward()
    ref = {k: to_f64(v) for k, v in kw.items()}
    f = lambda p: sum((a * to_f64(b)).sum() for a, b in zip(olm.block_norm(**p), (dr, dn)))   # noqa: E731
    rng = np.random.default_rng(0)
    for name, leaf in leaves.items():
        dy = rng.standard_normal(ref[name].shape)
        diff = (f({**ref, name: ref[name] + 1e-6 * dy}) - f({**ref, name: ref[name] - 1e-6 * dy})) / 2e-6
        got = (to_f64(leaf.grad) * dy).sum()
        assert abs(got - diff) <= 1e-4 * max(1.0, abs(diff)), name
    # the norm before the first block: r is the stream itself
    y = torch.randn(4, 20, device="cuda", requires_grad=True)
    r, n = prn.block_norm_apply(y, w_pre=leaves["w_pre"])
    assert r is y
    n.sum().backward()
    assert torch.equal(y.grad, prn.block_norm_backward(None, torch.ones_like(n), y.detach(), w_pre=kw["w_pre"])[0])
    # only r is used
    y.grad = None
    r, n = prn.block_norm_apply(y, dr[:4], w_pre=kw["w_pre"])
    r.sum().backward()
    assert torch.equal(y.grad, torch.ones_like(y))


def test_another_stream_and_a_graph():
    kw, dr, dn = _inputs(200, 128, "bf16", FULL, 8)
    h, x = kw.pop("h"), kw.pop("x")
    s = torch.cuda.Stream()
    want = prn.block_norm(h, x, **kw) + prn.block_norm_backward(dr, dn, h, x, **kw)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = prn.block_norm(h, x, **kw) + prn.block_norm_backward(dr, dn, h, x, **kw)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = prn.block_norm(h, x, **kw) + prn.block_norm_backward(dr, dn, h, x, **kw)
    for _ in range(3):
        h.normal_()
        dn.normal_()
        graph.replay()
        torch.cuda.synchronize()
        want = prn.block_norm(h, x, **kw) + prn.block_norm_backward(dr, dn, h, x, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype,d", [("bf16", 513), ("bf16", 519), ("bf16", 1025), ("bf16", 2049), ("bf16", 4099), ("bf16", 8185),
                                     ("bf16", 1001), ("f32", 515), ("f32", 769), ("f32", 1025), ("f32", 2051), ("f32", 513)])
@pytest.mark.parametrize("N", [3, 2500])
def test_in_place_at_widths_whose_last_chunk_crosses_waves(N, d, dtype):
    """The moved-back last chunk of a row reads channels of another wave: with no norm of h there is no sum, and
    so no barrier, between reading the row and writing r over it, unless the kernel puts one there."""
    kw, _, _ = _inputs(N, d, dtype, FULL, N + d)
    h, x = kw.pop("h"), kw.pop("x")
    for parts in ((), ("gate",), ("alpha",), ("w_pre",), ("gate", "alpha", "w_pre"), ("gate", "w_post", "w_pre")):
        p = {k: kw[k] if k in parts else None for k in kw}
        g, weights = p.pop("gate"), p
        n = None if weights["w_pre"] is None else torch.empty_like(h)
        want = prn.block_norm(h, x, gate=g, **weights)
        for over in ("h", "x"):
            hh, xx = h.clone(), x.clone()
            r = hh if over == "h" else xx
            B.prn_block_norm(hh, g, xx, r, n, **weights)
            assert torch.equal(r, want[0]) and (n is None or torch.equal(n, want[1])), (parts, over)
            if n is not None:      # n over the other input
                hh, xx = h.clone(), x.clone()
                r, m = (hh, xx) if over == "h" else (xx, hh)
                B.prn_block_norm(hh, g, xx, r, m, **weights)
                assert torch.equal(r, want[0]) and torch.equal(m, want[1]), (parts, over)


def test_the_norm_before_the_first_block_copies_nothing():
    """n is all that the differentiable form allocates: the stream goes on as it is."""
    y, w = torch.randn(4096, 512, device="cuda", requires_grad=True), torch.ones(512, device="cuda")
    prn.block_norm_apply(y, w_pre=w)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    r, n = prn.block_norm_apply(y, w_pre=w)
    assert r is y and torch.cuda.max_memory_allocated() - before < 1.5 * y.numel() * 4
    (n * 2).sum().backward()
    assert torch.equal(y.grad, prn.block_norm_backward(None, torch.full_like(n, 2.0), y.detach(), w_pre=w)[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-18, 1e-19, 1e-20])
def test_rows_whose_squares_leave_the_normal_range(size, dtype):
    """eps = 0: the mean of the squares is below 2^-126, where each square is off by half a step of 2^-149 (relative
    to the mean: 2^-150 / mean, halved by the root), and its root is not."""
    d = 96
    kw, _, dn = _inputs(5, d, dtype, (False, False, True, False, False), 11)
    h = (kw["h"].float() * size).to(TORCH_DT[dtype])
    u, h64 = torch.finfo(TORCH_DT[dtype]).eps / 2, to_f64(h)
    n = prn.block_norm(h, w_pre=kw["w_pre"], eps=0.0)[1]
    ref = olm.block_norm(h64, w_pre=to_f64(kw["w_pre"]), eps=0.0)[1]
    mean = (h64 ** 2).mean(-1, keepdims=True)
    rel = 160 * E24 + 2.0 ** -150 / mean
    assert (np.abs(to_f64(n) - ref) <= (u + rel) * np.abs(ref)).all()
    dh = prn.block_norm_backward(None, dn, h, w_pre=kw["w_pre"], eps=0.0)[0]
    args = (None, to_f64(dn), h64)
    ref = olm.block_norm_backward(*args, w_pre=to_f64(kw["w_pre"]), eps=0.0)["dh"]
    band = olm.block_norm_backward(*args, w_pre=to_f64(kw["w_pre"]), eps=0.0, size=True)["dh"]
    assert (np.abs(to_f64(dh) - ref) <= u * np.abs(ref) + 4 * rel * band).all()
