"""The vocabulary loss where its 16-bit terms could run out of range: tokens of
very unequal weight or size, products below fp32's range, several pieces of
two-term gradients, and the one fp16 rounding of bf16 data's dz.

Bands, first-order, per element, e = 2^-24, u = half a step of the storage
type, A = |x| |W|^T, g_n = max(|dloss_n|, |dloss_n + dlse_n|):
  operands  x is held to 2^-39 of its token's largest value, W to 2^-39 of the
            tensor's (a largest value of 2^14 .. 2^15 and half a step of 2^-24);
            above that bf16 data exactly, fp32 data to 2^-22 of itself, which
            the logits' count has
  logits    bz = (2 d + 8) e s A (fp32 data 12 d + 8) + s times the operands' floors
  lse       max bz of the row + (V / 2 + 64) e + 8 e (|lse| + max|z|)
  loss      lse's band + the target's logit's
  dz        relative 2^-11 (bf16 data: one fp16 rounding) or 4 e (two terms);
            2^-38 s g_n (half a step of 2^-24 over 2^13); p's exponent: bz + lse's
            band + 4 e (|z| + |lse|) + 16 e, against q = s (|dloss + dlse| p + |dloss| onehot)
  dx        u |dx| + sum of dz's band |W| + 2 (V + 64) e sum q |W| + W's floor sum q
  dW        u |dW| + sum of dz's band |x| + 2 (N + 64) e sum q |x|, and x, in it times
            a power of two in (g_n / 2, g_n], is held to 2^-39 max(g_n |x|): 2^-38 max(g_n |x|) sum q / g_n
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


def _inputs(N, V, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TORCH_DT[dtype]
    W = torch.randn(V, d, generator=g, device="cuda") / d ** 0.5
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    x = torch.randn(N, d, generator=g, device="cuda") + 4 * W[t]
    t[torch.rand(N, generator=g, device="cuda") < 0.1] = -100
    dloss = torch.rand(N, generator=g, device="cuda") + 0.5
    dlse = 0.1 * torch.randn(N, generator=g, device="cuda")
    return x.to(dt), W.to(dt), t, dloss, dlse


def _bands(x, W, t, dloss, dlse, dtype, scale):
    """(loss, lse, dx, dW) of the oracle and their bands."""
    (N, d), V = x.shape, W.shape[0]
    u = torch.finfo(TORCH_DT[dtype]).eps / 2
    loss, lse, z = olm.vocab_loss(x, W, t, scale)
    fx, fW = 2.0 ** -39 * np.abs(x).max(-1), 2.0 ** -39 * np.abs(W).max()
    bz = np.abs(x) @ np.abs(W).T
    bz *= ((2 * d + 8) if dtype == "bf16" else (12 * d + 8)) * E * scale
    bz += scale * (fx[:, None] * np.abs(W).sum(1)[None, :] + fW * np.abs(x).sum(1)[:, None])
    b_lse = bz.max(-1) + (V / 2 + 64) * E + 8 * E * (np.abs(lse) + np.abs(z).max(-1))
    at, rows = np.where((t >= 0) & (t < V), t, 0), np.arange(N)
    b_loss = b_lse + bz[rows, at] + 8 * E * np.abs(z[rows, at])
    dz = olm.vocab_loss_dz(dloss, dlse, z, lse, t, scale)
    one = np.where(t == -100, 0.0, dloss)
    both = one if dlse is None else one + dlse
    g = np.maximum(np.abs(one), np.abs(both))
    q = np.exp(z - lse[:, None]) * np.abs(both)[:, None]
    b_dz = (bz + b_lse[:, None] + 4 * E * (np.abs(z) + np.abs(lse)[:, None]) + 16 * E) * q
    q[rows, at] += np.abs(one)
    b_dz[rows, at] += 16 * E * np.abs(one)
    b_dz += (2.0 ** -11 if dtype == "bf16" else 4 * E) * np.abs(dz) / scale + 2.0 ** -38 * g[:, None]
    b_dz, q = scale * b_dz, scale * q
    dx, dW = dz @ W, dz.T @ x
    b_dx = u * np.abs(dx) + b_dz @ np.abs(W) + 2 * (V + 64) * E * (q @ np.abs(W)) + fW * q.sum(-1)[:, None]
    inv = np.divide(1.0, g, out=np.zeros_like(g), where=g > 0)
    b_dW = u * np.abs(dW) + b_dz.T @ np.abs(x) + 2 * (N + 64) * E * (q.T @ np.abs(x))
    b_dW += 2.0 ** -38 * (g * np.abs(x).max(-1)).max() * (q.T @ inv)[:, None]
    return (loss, lse, dx, dW), (b_loss, b_lse, b_dx, b_dW)


def _check(x, W, t, dloss, dlse, dtype, scale=1.0, names=("loss", "lse", "dx", "dW"), rows=None):
    """Every output in its band; of `names` only, and of the tokens `rows` only (not for dW)."""
    loss, lse = prn.vocab_loss(x, W, t, scale=scale)
    dx, dW = prn.vocab_loss_backward(dloss, x, W, t, lse, dlse=dlse, scale=scale)
    ref, band = _bands(to_f64(x), to_f64(W), t.cpu().numpy(), to_f64(dloss), None if dlse is None else to_f64(dlse), dtype, scale)
    for name, got, r, b in zip(("loss", "lse", "dx", "dW"), (loss, lse, dx, dW), ref, band):
        if name not in names:
            continue
        part = slice(None) if rows is None or name == "dW" else rows
        err = np.abs(to_f64(got) - r)[part] / np.maximum(b[part], 1e-300)
        worst = float(np.nan_to_num(err, nan=np.inf).max())
        say(f"  {name}: of the band {worst:.3g}")
        assert worst <= 1.0, name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,d", [(64, 128, 64), (65, 129, 65), (2, 5000, 40), (257, 2048, 256), (700, 513, 129)])
def test_dz_is_rounded_once_to_fp16(N, V, d, dtype):
    say(f"[case] vocab loss N={N} V={V} d={d} {dtype}")
    _check(*_inputs(N, V, d, dtype, N + V), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("with_dlse", [False, True])
def test_tokens_of_unequal_weight(dtype, with_dlse):
    """dloss from 1 down to 1e-12, and one token without any: every row of dx is as good as alone."""
    x, W, t, dloss, dlse = _inputs(260, 700, 48, dtype, 1)
    w = 10.0 ** -(torch.arange(260, device="cuda") % 13).float()
    w[7] = 0
    _check(x, W, t, dloss * w, dlse * w if with_dlse else None, dtype)
    _check(x, W, t, -dloss * w * 2.0 ** 20, dlse * w if with_dlse else None, dtype, scale=0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_large_token_leaves_the_others(dtype):
    x, W, t, dloss, dlse = _inputs(140, 200, 64, dtype, 2)
    x[3] *= 2.0 ** 44
    rows = np.arange(140) != 3
    _check(x, W, t, dloss, dlse, dtype, names=("loss", "lse", "dx"), rows=rows)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sx,sw", [(1e-20, 1e-20), (1e-30, 1e-12), (1e-38, 1.0), (0.0, 1e-30), (1e-36, 1e-36)])
def test_logits_below_the_range(dtype, sx, sw):
    """The logits are zero but for what fp32 cannot hold: the loss is log V."""
    x, W, t, dloss, dlse = _inputs(70, 300, 40, dtype, 3)
    x, W = x * sx, W * sw
    loss, lse = prn.vocab_loss(x, W, t)
    assert (np.abs(to_f64(lse) - np.log(300)) <= (150 + 64) * E + 8 * E * 6).all()
    assert torch.equal(loss[t != -100], lse[t != -100])
    dx, dW = prn.vocab_loss_backward(dloss, x, W, t, lse, dlse=dlse)
    assert dx.isfinite().all() and dW.isfinite().all()


@pytest.mark.parametrize("N,V", [(9000, 16001), (66000, 2100)])
def test_several_pieces_of_two_terms(N, V):
    """More than 512 MB of fp32 data's dz: dx adds up over pieces, the last one short and of no multiple of 8; in the
    second case 258 row tiles, the last two's sums in slices."""
    whole = N * V * 4
    assert B.prn_vocab_loss_backward_workspace_bytes(torch.float32, N, V, 16) < whole
    say(f"[case] vocab loss N={N} V={V} f32, several pieces")
    _check(*_inputs(N, V, 16, "f32", 4), "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite(dtype, bad):
    """In x: in their tokens' rows, and in dW; in W: in every token whose logit of it is not -inf."""
    x, W, t, dloss, dlse = _inputs(150, 200, 40, dtype, 5)
    t[20] = -100
    loss, lse = prn.vocab_loss(x, W, t)
    dx, _ = prn.vocab_loss_backward(dloss, x, W, t, lse, dlse=dlse)
    y = x.clone()
    y[9, 3] = y[20, 0] = bad
    rows = torch.zeros(150, dtype=torch.bool, device="cuda")
    rows[9] = rows[20] = True
    loss2, lse2 = prn.vocab_loss(y, W, t)
    dx2, dW2 = prn.vocab_loss_backward(dloss, y, W, t, lse2, dlse=dlse)
    assert loss2[20] == 0 and not loss2[9].isfinite() and not lse2[rows].isfinite().any()
    assert torch.equal(loss2[~rows], loss[~rows]) and torch.equal(lse2[~rows], lse[~rows])
    assert dx2[rows].isnan().all() and torch.equal(dx2[~rows], dx[~rows]) and dW2.isnan().all()
    U = W.clone()
    U[30, 5] = bad
    loss3, lse3 = prn.vocab_loss(x, U, t)
    high = ~(x[:, 5] * bad == -float("inf"))
    assert not lse3[high].isfinite().any() and not loss3[high & (t != -100)].isfinite().any()
    if dtype == "bf16":   # the others have no share of entry 30
        keep = torch.arange(200, device="cuda") != 30
        _, want, z = olm.vocab_loss(to_f64(x), to_f64(W[keep]), np.full(150, -100))
        size = (np.abs(to_f64(x)) @ np.abs(to_f64(W[keep])).T).max(-1)
        band = (2 * 40 + 8) * E * size + (100 + 64) * E + 8 * E * (np.abs(want) + np.abs(z).max(-1))
        assert (np.abs(to_f64(lse3) - want) <= band)[~high.cpu().numpy()].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V", [(64, 1000), (300, 3000)])
@pytest.mark.parametrize("size", [80.0, 100.0, 1e3, 1e5, 1e7, 2e9, 1e12, 1e18])
def test_logits_far_from_zero(dtype, N, V, size):
    """All of a token's logits around -size or size, or spread over that: loss and lse against the oracle.  The
    tokens beside them in a wave are ordinary ones."""
    x, W, t, _, _ = _inputs(N, V, 40, dtype, 7)
    W[:, 0] = 1.0
    x[0:60:4, 0] = -size
    x[1:60:4, 0] = size
    x[2:60:4] *= size
    loss, lse = prn.vocab_loss(x, W, t)
    (ref, ref_lse, _, _), (b_loss, b_lse, _, _) = _bands(to_f64(x), to_f64(W), t.cpu().numpy(), np.ones(N), None, dtype, 1.0)
    for name, got, r, b in (("loss", loss, ref, b_loss), ("lse", lse, ref_lse, b_lse)):
        worst = np.nan_to_num(np.abs(to_f64(got) - r) / b, nan=np.inf).max()
        say(f"  {name}: of the band {worst:.3g}")
        assert worst <= 1.0, name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 24, 2.0 ** 27, 2.0 ** 32, 2.0 ** 44])
@pytest.mark.parametrize("shift", [False, True])
def test_logits_that_hold_no_fraction(dtype, size, shift):
    """Logits of 1e7 and more, of either sign, or (shift) all of a token's the same: a probability of one entry is at
    most 1 whatever its exponent's rounding, so dx and dW stay finite and dx within what its coefficients allow;
    with fp32 data, whose logits are the same bits both ways, it is that of the one entry that counts."""
    x, W, t, dloss, dlse = _inputs(150, 200, 64, dtype, 6)
    W[:, 0] = -1.0
    if shift:
        x[5:9, 0] = size        # every logit far below zero, their differences lost
        x[9:12, 0] = -size
    else:
        x[5:12] *= size
    loss, lse = prn.vocab_loss(x, W, t)
    dx, dW = prn.vocab_loss_backward(dloss, x, W, t, lse, dlse=dlse)
    assert loss.isfinite().all() and lse.isfinite().all() and dx.isfinite().all() and dW.isfinite().all()
    W64 = to_f64(W)
    one = np.where(t.cpu().numpy() == -100, 0.0, to_f64(dloss))
    both = one + to_f64(dlse)
    if shift:   # up to 200 entries of up to twice their coefficient's power of two each
        bound = (200 * 4 + 1) * np.maximum(np.abs(one), np.abs(both))[5:12, None] * np.abs(W64).max(0)
        assert (np.abs(to_f64(dx)[5:12]) <= bound).all()
        return
    z = to_f64(x) @ W64.T
    top = np.sort(z, -1)
    A = (np.abs(to_f64(x)) @ np.abs(W64).T).max(-1)
    alone = top[:, -1] - top[:, -2] > (12 * 64 + 8) * E * A * 2 + 40     # the largest stands out of the logits' errors
    want = both[:, None] * W64[z.argmax(-1)] - np.where((t.cpu().numpy() >= 0), one, 0.0)[:, None] * W64[t.cpu().numpy().clip(0)]
    rows = [n for n in range(5, 12) if alone[n]]
    if dtype == "f32" and size >= 2.0 ** 32:   # lse is the largest logit, without a fraction
        assert rows
        size_ = (np.abs(both) + np.abs(one))[:, None] * np.abs(W64).max(0)
        assert (np.abs(to_f64(dx) - want) <= 2.0 ** -20 * size_)[rows].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mask", [-1e9, -1e30, -3.3895314e38])
@pytest.mark.parametrize("N,V,d", [(64, 700, 40), (150, 1500, 300), (5, 9000, 600)])
def test_masked_entries(N, V, d, mask, dtype):
    """A channel of ones in x and of a bias in W, which is a mask's value at some entries (-1e9, or the type's
    lowest): their probability is 0, and no other entry, token or channel feels how large it is.  The bands are
    those of the entries that are left, over the other channels."""
    x, W, t, dloss, dlse = _inputs(N, V, d, dtype, 8)
    x[:, 0] = 1.0
    off = torch.zeros(V, dtype=torch.bool, device="cuda")
    off[torch.randperm(V, generator=torch.Generator().manual_seed(V))[: V // 5].cuda()] = True
    t = torch.where(off[t.clamp(min=0)], torch.full_like(t, -100), t)
    W[off, 0] = mask
    loss, lse = prn.vocab_loss(x, W, t)
    dx, dW = prn.vocab_loss_backward(dloss, x, W, t, lse, dlse=dlse)
    keep = (~off).cpu().numpy()
    new = np.where(keep, np.cumsum(keep) - 1, 0)
    tn = t.cpu().numpy()
    ref, band = _bands(to_f64(x), to_f64(W)[keep], np.where(tn < 0, -100, new[tn.clip(0)]), to_f64(dloss), to_f64(dlse), dtype, 1.0)
    for name, got, r, b in zip(("loss", "lse", "dx", "dW"), (loss, lse, dx[:, 1:], dW[~off]), ref, band):
        r, b = (r[:, 1:], b[:, 1:]) if name == "dx" else (r, b)
        worst = np.nan_to_num(np.abs(to_f64(got) - r) / b, nan=np.inf).max()
        say(f"  {name}: of the band {worst:.3g}")
        assert worst <= 1.0, name
    assert not dW[off].any() and dx.isfinite().all()


@pytest.mark.parametrize("seed", range(48))
def test_seeded_sweep(seed):
    """Sizes, types, scales and data of every kind above, drawn."""
    r = np.random.default_rng(seed)
    dtype = ("bf16", "f32")[int(r.integers(2))]
    N, V, d = (int(2 ** r.uniform(0, top)) for top in (10, 12, 9.3))
    x, W, t, dloss, dlse = _inputs(N, V, d, dtype, seed)
    scale, kind = 1.0, ("plain", "offset", "weights", "rows", "entries", "scale", "large")[seed % 7]
    spread = lambda n: 10.0 ** (-8 * torch.from_numpy(r.random((n, 1))).float().cuda())   # noqa: E731
    if kind == "offset":
        W[:, 0] = 1.0
        x[::2, 0] = float(r.choice([-1, 1]) * 10 ** r.uniform(1, 4))
    elif kind == "weights":
        w = spread(N)[:, 0]
        dloss, dlse = dloss * w, dlse * w
    elif kind == "rows":
        x = (x.float() * spread(N)).to(x.dtype)
    elif kind == "entries":
        W = (W.float() * spread(V)).to(W.dtype)
    elif kind == "scale":
        scale = float(10 ** r.uniform(-3, 1))
    elif kind == "large":
        x = x * float(r.choice([10, 100]))
    say(f"[case] {seed} {kind} N={N} V={V} d={d} {dtype} scale={scale:.3g}")
    _check(x, W, t, dloss, dlse if r.integers(2) else None, dtype, scale=scale)
