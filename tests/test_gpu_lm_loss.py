"""GPU parity of the vocabulary loss and its gradients against oracle.lm.

Bands, first-order, per element, e = 2^-24, u = half a step of the storage
type, A = |x| |W|^T (the size of a logit's products):
  logits  dz_ = (2 d + 8) e s A: d fp32 additions of exact products (two
          roundings each allowed for the matrix cores' order); fp32 data, whose
          values go as two terms good to 2^-22 each: 12 d + 8 instead
  lse     max dz_ of the row + (V / 2 + 64) e (sums of positive terms) + 8 e (|lse| + max|z|)
  loss    lse's band + the target's logit's
  dz      relative 2^-8 (one rounding to 8 bits; bf16 storage only) + the error of
          p's exponent: dz_ + lse's band + 4 e (|z| + |lse|) + 16 e, against
          q = s (|dloss + dlse| p + |dloss| onehot)
  dx      u |dx| + sum of dz's band |W| + 2 (V + 64) e sum q |W|; dW likewise with N
"""
import numpy as np
import pytest
import torch

import nonlinear_rnn_amd as prn
from gpu_helpers import TORCH_DT, say, to_f64
from nonlinear_rnn_amd import binding as B
from oracle import lm as olm

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


def _inputs(N, V, d, dtype, seed, ids=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TORCH_DT[dtype]
    W = torch.randn(V, d, generator=g, device="cuda") / d ** 0.5
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    x = torch.randn(N, d, generator=g, device="cuda") + 4 * W[t]
    t[torch.rand(N, generator=g, device="cuda") < 0.1] = -100
    dloss = torch.rand(N, generator=g, device="cuda") + 0.5
    dlse = 0.1 * torch.randn(N, generator=g, device="cuda")
    return x.to(dt), W.to(dt), t.to(ids), dloss, dlse


def _bands(x, W, t, dloss, dlse, dtype, scale):
    """(loss, lse, dx, dW) of the oracle and their bands."""
    N, d = x.shape
    V = W.shape[0]
    u = torch.finfo(TORCH_DT[dtype]).eps / 2
    loss, lse, z = olm.vocab_loss(x, W, t, scale)
    A = np.abs(x) @ np.abs(W).T
    bz = ((2 * d + 8) if dtype == "bf16" else (12 * d + 8)) * E * scale * A
    b_lse = bz.max(-1) + (V / 2 + 64) * E + 8 * E * (np.abs(lse) + np.abs(z).max(-1))
    at = np.where((t >= 0) & (t < V), t, 0)
    rows = np.arange(N)
    b_loss = b_lse + bz[rows, at] + 8 * E * np.abs(z[rows, at])
    dz = olm.vocab_loss_dz(dloss, dlse, z, lse, t, scale)
    one = np.where(t == -100, 0.0, np.abs(dloss))
    p = np.exp(z - lse[:, None])
    q = p * np.abs(np.where(t == -100, 0.0, dloss) + (0.0 if dlse is None else dlse))[:, None]
    rel = bz + b_lse[:, None] + 4 * E * (np.abs(z) + np.abs(lse)[:, None]) + 16 * E
    b_dz = rel * q
    q[rows, at] += one
    b_dz[rows, at] += 16 * E * one
    b_dz += (2.0 ** -8 if dtype == "bf16" else 3 * E) * np.abs(dz) / scale
    b_dz, q = scale * b_dz, scale * q
    dx, dW = dz @ W, dz.T @ x
    b_dx = u * np.abs(dx) + b_dz @ np.abs(W) + 2 * (V + 64) * E * (q @ np.abs(W))
    b_dW = u * np.abs(dW) + b_dz.T @ np.abs(x) + 2 * (N + 64) * E * (q.T @ np.abs(x))
    return (loss, lse, dx, dW), (b_loss, b_lse, b_dx, b_dW)


def _check(N, V, d, dtype, scale=1.0, with_dlse=True, ids=torch.int64, seed=0):
    say(f"[case] vocab loss N={N} V={V} d={d} {dtype} scale={scale} {ids}")
    x, W, t, dloss, dlse = _inputs(N, V, d, dtype, N + V + d + seed, ids)
    dlse = dlse if with_dlse else None
    loss, lse = prn.vocab_loss(x, W, t, scale=scale)
    dx, dW = prn.vocab_loss_backward(dloss, x, W, t, lse, dlse=dlse, scale=scale)
    ref, band = _bands(to_f64(x), to_f64(W), t.cpu().numpy().astype(np.int64), to_f64(dloss),
                       None if dlse is None else to_f64(dlse), dtype, scale)
    for name, got, r, b in zip(("loss", "lse", "dx", "dW"), (loss, lse, dx, dW), ref, band):
        err = np.abs(to_f64(got) - r)
        worst = float((err / np.maximum(b, 1e-300)).max())
        say(f"  {name}: max error {err.max():.2e}, of the band {worst:.2f}")
        assert worst <= 1.0, name
    assert (loss[t == -100] == 0).all()
    again = prn.vocab_loss(x, W, t, scale=scale) + prn.vocab_loss_backward(dloss, x, W, t, lse, dlse=dlse, scale=scale)
    assert all(torch.equal(a, b) for a, b in zip((loss, lse, dx, dW), again))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,d", [
    (1, 1, 1), (1, 2, 8), (3, 31, 7), (5, 33, 20), (64, 128, 64), (63, 127, 63), (65, 129, 65), (64, 1000, 512),
    (2, 5000, 40), (128, 256, 32), (130, 257, 100), (129, 300, 520), (300, 999, 24), (257, 2048, 256), (700, 513, 129),
    (1100, 3001, 48)])
def test_vocab_loss_matches_oracle(N, V, d, dtype):
    _check(N, V, d, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scale_int32_targets_and_no_gradient_of_lse(dtype):
    _check(200, 700, 96, dtype, scale=3.0, with_dlse=False, ids=torch.int32)
    _check(40, 700, 96, dtype, scale=0.05)


@pytest.mark.parametrize("dtype,N,V", [("bf16", 9000, 31000), ("f32", 6000, 8000)])
def test_several_pieces_of_the_vocabulary(dtype, N, V):
    """dz of the whole vocabulary exceeds the workspace's piece (256 MB): dx adds up over pieces."""
    _check(N, V, 16, dtype)


@pytest.mark.parametrize("dtype,N,V", [("bf16", 1030, 66000), ("f32", 1030, 66000), ("bf16", 66000, 1030)])
def test_rest_of_the_rounds_in_slices(dtype, N, V):
    """258 row tiles: 256 over the whole sum, the sum of the last two in slices (of dW, or of dx)."""
    _check(N, V, 16, dtype)


def test_rows_without_a_loss_and_targets_out_of_range():
    x, W, t, dloss, dlse = _inputs(150, 300, 40, "f32", 1)
    t[:] = -100                                     # nothing to learn from
    loss, lse = prn.vocab_loss(x, W, t)
    dx, dW = prn.vocab_loss_backward(dloss, x, W, t, lse)
    assert not loss.any() and not dx.any() and not dW.any()
    t = torch.randint(0, 300, (150,), device="cuda")
    good = prn.vocab_loss(x, W, t)[0]
    t2 = t.clone()
    t2[5], t2[100] = 300, -1
    loss, lse = prn.vocab_loss(x, W, t2)
    bad = torch.zeros(150, dtype=torch.bool, device="cuda")
    bad[5] = bad[100] = True
    assert loss[bad].isnan().all() and torch.equal(loss[~bad], good[~bad])
    dx, dW = prn.vocab_loss_backward(dloss, x, W, t2, lse)
    assert dx[bad].isnan().all() and not dx[~bad].isnan().any() and dW.isnan().all()
    # another ignore index, one that is a row of the table
    loss = prn.vocab_loss(x, W, t, ignore_index=int(t[7]))[0]
    assert loss[7] == 0 and torch.equal(loss[t != t[7]], good[t != t[7]])


def test_large_logits_and_bad_values_stay_in_their_rows():
    x, W, t, dloss, _ = _inputs(140, 400, 64, "f32", 2)
    x[3] *= 1e4                                     # logits in the tens of thousands
    loss, lse = prn.vocab_loss(x, W, t)
    ref = olm.vocab_loss(to_f64(x), to_f64(W), t.cpu().numpy())
    size = np.abs(to_f64(x)) @ np.abs(to_f64(W)).T
    assert (np.abs(to_f64(lse) - ref[1]) <= (12 * 64 + 400) * E * size.max(-1) + 400 * E).all()
    dx, dW = prn.vocab_loss_backward(dloss, x, W, t, lse)
    assert dx.isfinite().all() and dW.isfinite().all()
    y = x.clone()
    y[9] = float("nan")
    l2, s2 = prn.vocab_loss(y, W, t)
    keep = torch.arange(140, device="cuda") != 9
    assert s2[9].isnan() and torch.equal(s2[keep], lse[keep]) and torch.equal(l2[keep], loss[keep])
    dx2 = prn.vocab_loss_backward(dloss, y, W, t, s2, want_W=False)[0]
    assert dx2[9].isnan().all() and torch.equal(dx2[keep], dx[keep])


def test_values_far_below_the_largest():
    """fp32 rows from 1 down to 1e-9 of the largest value: on top of the usual band the operands may be off by
    2^-39 of their tensor's largest value (two fp16 terms in units of that value)."""
    N, V, d = 160, 200, 48
    x, W, t, dloss, _ = _inputs(N, V, d, "f32", 12)
    x *= 10.0 ** -(torch.arange(N, device="cuda") % 10)[:, None].float()
    W *= 10.0 ** -(torch.arange(V, device="cuda") % 7)[:, None].float()
    loss, lse = prn.vocab_loss(x, W, t)
    dx, dW = prn.vocab_loss_backward(dloss, x, W, t, lse)
    x64, W64, tn, dl = to_f64(x), to_f64(W), t.cpu().numpy(), to_f64(dloss)
    ref, band = _bands(x64, W64, tn, dl, None, "f32", 1.0)
    ux, uw = 2.0 ** -39 * np.abs(x64).max(), 2.0 ** -39 * np.abs(W64).max()
    bz = (ux * np.abs(W64).sum(1)[None, :] + uw * np.abs(x64).sum(1)[:, None])
    one = np.where(tn == -100, 0.0, np.abs(dl))
    dz = 2 * one[:, None] * bz            # through p and the target's entry
    u = 2.0 ** -39 * one.max()            # dz's own terms
    extra = (2 * bz.max(-1), bz.max(-1), dz @ np.abs(W64) + u * np.abs(W64).sum(0) + uw * 2 * one[:, None],
             dz.T @ np.abs(x64) + u * np.abs(x64).sum(0) + ux * 2 * one.sum())
    for name, got, r, b, e in zip(("loss", "lse", "dx", "dW"), (loss, lse, dx, dW), ref, band, extra):
        worst = float((np.abs(to_f64(got) - r) / (b + e)).max())
        say(f"  {name}: of the band {worst:.3f}")
        assert worst <= 1.0, name


def test_gradients_that_are_zero_or_one_sided():
    x, W, t, dloss, dlse = _inputs(90, 200, 24, "bf16", 3)
    loss, lse = prn.vocab_loss(x, W, t)
    dx, dW = prn.vocab_loss_backward(torch.zeros_like(dloss), x, W, t, lse)
    assert not dx.any() and not dW.any()
    full = prn.vocab_loss_backward(dloss, x, W, t, lse, dlse=dlse)
    assert torch.equal(prn.vocab_loss_backward(dloss, x, W, t, lse, dlse=dlse, want_W=False)[0], full[0])
    only = prn.vocab_loss_backward(dloss, x, W, t, lse, dlse=dlse, want_x=False)
    assert only[0] is None and torch.equal(only[1], full[1])
    # coefficients far below 1, as of a mean over many tokens: the result scales with them
    tiny = prn.vocab_loss_backward(dloss * 2.0 ** -40, x, W, t, lse, dlse=dlse * 2.0 ** -40)
    assert torch.equal(tiny[0].float() * 2.0 ** 40, full[0].float()) and torch.equal(tiny[1].float() * 2.0 ** 40, full[1].float())


def test_empty_strided_and_misaligned():
    x, W, t, dloss, _ = _inputs(60, 210, 48, "bf16", 4)
    loss, lse = prn.vocab_loss(x, W, t)
    back = prn.vocab_loss_backward(dloss, x, W, t, lse)
    l3, s3 = prn.vocab_loss(x.view(3, 20, 48), W, t.view(3, 20))
    assert l3.shape == (3, 20) and torch.equal(l3.view(-1), loss) and torch.equal(s3.view(-1), lse)
    wide = torch.zeros(60, 60, device="cuda", dtype=x.dtype)
    wide[:, 5:53] = x
    assert torch.equal(prn.vocab_loss(wide[:, 5:53], W, t)[0], loss)
    flat = torch.empty(210 * 48 + 1, device="cuda", dtype=x.dtype)
    flat[1:] = W.view(-1)
    off = flat[1:].view(210, 48)
    assert torch.equal(prn.vocab_loss(x, off, t)[0], loss)
    assert torch.equal(prn.vocab_loss_backward(dloss, x, off, t, lse)[1], back[1])
    with pytest.raises(B.PrnError, match="16-byte"):
        B.prn_vocab_loss(x, off, t, loss.clone(), lse.clone())
    e = prn.vocab_loss(x[:0], W, t[:0])
    assert e[0].shape == e[1].shape == (0,)
    dx, dW = prn.vocab_loss_backward(dloss[:0], x[:0], W, t[:0], lse[:0])
    assert dx.shape == (0, 48) and dW.shape == W.shape and not dW.any()


def test_autograd_against_differences():
    x, W, t, dloss, dlse = _inputs(12, 30, 10, "f32", 5)
    x, W = x.requires_grad_(), W.requires_grad_()
    loss, lse = prn.vocab_loss_apply(x, W, t, scale=0.5)
    ((loss * dloss).sum() + (lse * dlse).sum()).backward()
    x64, W64, tn = to_f64(x), to_f64(W), t.cpu().numpy()

    def f(x, W):
        a, b, _ = olm.vocab_loss(x, W, tn, 0.5)
        return (a * to_f64(dloss)).sum() + (b * to_f64(dlse)).sum()

    rng = np.random.default_rng(0)
    for leaf, y, g in ((x, x64, lambda y: f(y, W64)), (W, W64, lambda y: f(x64, y))):
        dy = rng.standard_normal(y.shape)
        diff = (g(y + 1e-6 * dy) - g(y - 1e-6 * dy)) / 2e-6
        assert abs((to_f64(leaf.grad) * dy).sum() - diff) <= 1e-4 * max(1.0, abs(diff))
    # a head that is frozen, and only lse used
    W2 = W.detach()
    x.grad = None
    prn.vocab_loss_apply(x, W2, t)[1].sum().backward()
    want = prn.vocab_loss_backward(torch.zeros(12, device="cuda"), x.detach(), W2, t, prn.vocab_loss(x.detach(), W2, t)[1],
                                   dlse=torch.ones(12, device="cuda"), want_W=False)[0]
    assert torch.equal(x.grad, want)


def test_another_stream_and_a_graph():
    x, W, t, dloss, _ = _inputs(200, 600, 64, "bf16", 6)
    run = lambda: (lambda a: a + prn.vocab_loss_backward(dloss, x, W, t, a[1]))(prn.vocab_loss(x, W, t))   # noqa: E731
    want = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        x.normal_()
        dloss.uniform_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, run()))


def test_more_tokens_than_one_row_of_a_grid():
    """2^26 tokens and a few: a wave each is more threads than one dimension of a launch may have."""
    x, W, t, _, _ = _inputs(1024, 16, 8, "bf16", 9)
    loss, lse = prn.vocab_loss(x, W, t)
    n = (1 << 16) + 1
    big = prn.vocab_loss(x.repeat(n, 1)[:-700], W, t.repeat(n)[:-700])
    for got, want in zip(big, (loss, lse)):
        assert torch.equal(got[:1024 * (n - 1)].view(n - 1, 1024), want.expand(n - 1, 1024))
        assert torch.equal(got[1024 * (n - 1):], want[:324])
