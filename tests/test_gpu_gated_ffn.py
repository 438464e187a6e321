"""The gated feed-forward product on the GPU against oracle.gated in float64.

Tolerances are the oracle's elementwise bounds (gated_ffn_bounds) and the
output's own rounding; the gradients of the sums are stored once in between.
"""
import numpy as np
import pytest
import torch

import nonlinear_rnn_amd as prn
from nonlinear_rnn_amd import binding as B
from oracle import gated

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def _np(t):
    return t.detach().double().cpu().numpy()


def _case(N, d, F, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    new = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    return new(N, d).to(dtype).cuda(), (new(2 * F, d) * (1.5 / d ** 0.5)).to(dtype).cuda(), new(N, F).to(dtype).cuda()


def _close(name, got, want, bound, dtype):
    got = _np(got)
    tol = bound * (1 + HALF[dtype]) + HALF[dtype] * np.abs(want) + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    worst = (np.abs(got - want) / tol).max() if got.size else 0.0
    print(f"  {name}: worst {worst:.3f} of its tolerance", flush=True)
    assert not bad.any(), (name, np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])


def _check(x, W, dout, kind, dtype):
    xd, Wd, gd = _np(x), _np(W), _np(dout)
    out = prn.gated_ffn(x, W, act=kind)
    dx, dW = prn.gated_ffn_backward(dout, x, W, act=kind)
    b_out, b_dx, b_dW = gated.gated_ffn_bounds(xd, Wd, kind, gd, HALF[dtype])
    want_dx, want_dW = gated.gated_ffn_backward(xd, Wd, gd, kind)
    _close("out", out, gated.gated_ffn(xd, Wd, kind), b_out, dtype)
    _close("dx", dx, want_dx, b_dx, dtype)
    _close("dW", dW, want_dW, b_dW, dtype)


SIZES = [(1, 1, 1), (1, 8, 32), (2, 7, 3), (3, 64, 31), (16, 128, 64), (17, 130, 65), (33, 40, 200), (64, 512, 96),
         (65, 100, 129), (127, 16, 64), (128, 64, 128), (129, 72, 130), (256, 256, 128), (300, 200, 100), (520, 24, 257),
         (1030, 96, 70)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["silu", "sigmoid"])
@pytest.mark.parametrize("N,d,F", SIZES)
def test_sizes(N, d, F, kind, dtype):
    _check(*_case(N, d, F, dtype, seed=N + d + F), kind, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,d,F", [(4096, 32, 1536), (5000, 40, 1300), (12800, 24, 520), (8200, 7, 515), (2500, 130, 1999),
                                   (33000, 16, 33)])
def test_large_tiles(N, d, F, dtype):
    _check(*_case(N, d, F, dtype), "silu", dtype)


@pytest.mark.parametrize("N,d,F", [(3, 64, 96), (65, 100, 129), (300, 72, 77), (1030, 96, 250), (2000, 31, 64)])
def test_bf16_gradients_of_few_tiles_round_once(N, d, F):
    """The gradients of the sums have two bf16 terms in between: off by 2^-16 of themselves, no more."""
    x, W, dout = _case(N, d, F, torch.bfloat16, seed=7)
    xd, Wd, gd = _np(x), _np(W), _np(dout)
    dx, dW = prn.gated_ffn_backward(dout, x, W)
    _, b_dx, b_dW = gated.gated_ffn_bounds(xd, Wd, "silu", gd, 2.0 ** -16)
    want_dx, want_dW = gated.gated_ffn_backward(xd, Wd, gd, "silu")
    _close("dx", dx, want_dx, b_dx, torch.bfloat16)
    _close("dW", dW, want_dW, b_dW, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_values_far_apart(dtype):
    """A large token, a large row of W, and zeros, each held to its own size."""
    x, W, dout = _case(100, 48, 40, dtype)
    x[3] *= 2.0 ** 20
    W[7] *= 2.0 ** 15
    x[5] = 0
    W[50] = 0
    dout[9] *= 2.0 ** -30
    dout[11] = 0
    _check(x, W, dout, "sigmoid", dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,F", [(5, 24), (150, 24), (2600, 1999)])
def test_what_is_not_finite_stays_in_its_row(dtype, N, F):
    x, W, dout = _case(N, 40, F, dtype)
    out, (dx, _) = prn.gated_ffn(x, W), prn.gated_ffn_backward(dout, x, W)
    for bad in (float("nan"), float("inf"), float("-inf")):
        y = x.clone()
        y[3, 5] = bad
        out2, (dx2, _) = prn.gated_ffn(y, W), prn.gated_ffn_backward(dout, y, W)
        rest = [n for n in range(N) if n != 3]
        assert torch.equal(out2[rest], out[rest]) and torch.equal(dx2[rest], dx[rest])
        assert not torch.isfinite(out2[3]).all()


def test_no_rows():
    x, W = torch.empty(0, 24, device="cuda"), torch.randn(16, 24, device="cuda")
    assert prn.gated_ffn(x, W).shape == (0, 8)
    dx, dW = prn.gated_ffn_backward(torch.empty(0, 8, device="cuda"), x, W)
    assert dx.shape == (0, 24) and (dW == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_shapes_layouts_and_the_same_bits(dtype):
    x, W, dout = _case(210, 36, 40, dtype)
    out, (dx, dW) = prn.gated_ffn(x, W), prn.gated_ffn_backward(dout, x, W)
    wide = torch.empty(210, 37, dtype=dtype, device="cuda")
    wide[:, 1:] = x
    Wt = W.t().contiguous().t()
    y, g = wide[:, 1:].unflatten(0, (3, 70)), dout.view(3, 70, 40)
    assert torch.equal(prn.gated_ffn(y, Wt), out.view(3, 70, 40))
    dx2, dW2 = prn.gated_ffn_backward(g, y, Wt)
    assert torch.equal(dx2, dx.view(3, 70, 36)) and torch.equal(dW2, dW)
    only = prn.gated_ffn_backward(dout, x, W, want_W=False)
    assert torch.equal(only[0], dx) and only[1] is None
    only = prn.gated_ffn_backward(dout, x, W, want_x=False)
    assert torch.equal(only[1], dW) and only[0] is None


def test_autograd():
    x, W, dout = _case(50, 24, 16, torch.float32)
    x.requires_grad_(), W.requires_grad_()
    dx, dW = torch.autograd.grad((prn.gated_ffn_apply(x, W, act="sigmoid") * dout).sum(), (x, W))
    want = prn.gated_ffn_backward(dout, x, W, act="sigmoid")
    assert torch.equal(dx, want[0]) and torch.equal(dW, want[1])
    g, = torch.autograd.grad(prn.gated_ffn_apply(x, W).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        g.square().sum().backward()


@pytest.mark.parametrize("N", [3, 400])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_captured_and_replayed(N, dtype):
    x, W, dout = _case(N, 52, 70, dtype)
    both = lambda: (prn.gated_ffn(x, W), *prn.gated_ffn_backward(dout, x, W))   # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for k in range(4):
        for t, new in zip((x, W, dout), _case(N, 52, 70, dtype, seed=k + 1)):
            t.copy_(new)
        want = [t.clone() for t in both()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), k


def test_refusals():
    x, W = torch.zeros(4, 8, device="cuda"), torch.zeros(6, 8, device="cuda")
    for bad in (W[:5], W[:, :4], W[0]):
        with pytest.raises(ValueError):
            prn.gated_ffn(x, bad)
    with pytest.raises(ValueError):
        prn.gated_ffn(x, W, act="tanh")
    with pytest.raises(TypeError):
        prn.gated_ffn(x, W.bfloat16())
    with pytest.raises(TypeError):
        prn.gated_ffn(x.half(), W.half())
    with pytest.raises(ValueError):
        prn.gated_ffn_backward(torch.zeros(3, 4, device="cuda"), x, W)   # rows and columns the wrong way round
    with pytest.raises(ValueError):
        prn.gated_ffn_backward(torch.zeros(4, 2, device="cuda"), x, W)
    assert B.lib() is not None


def test_offsets_past_32_bits():
    """2^20 + 77 rows of 2100 outputs: the last rows are those of a call of their own size."""
    N, d, F = 2 ** 20 + 77, 16, 2100
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()   # noqa: E731
    x, W, dout = new(N, d), new(2 * F, d), new(N, F)
    few = slice(N - 4096, N)   # of the same kind of tiles
    out = prn.gated_ffn(x, W)
    assert torch.equal(out[few], prn.gated_ffn(x[few].contiguous(), W))
    del out
    dx, _ = prn.gated_ffn_backward(dout, x, W, want_W=False)
    want, _ = prn.gated_ffn_backward(dout[few].contiguous(), x[few].contiguous(), W, want_W=False)
    # the sums may be cut in other slices: fp32 sums of 2 F products, and the result's rounding
    bound = HALF[torch.bfloat16] * want.double().abs() * 2 + 8 * F * 2.0 ** -24 * _magnitude(x[few], W, dout[few])
    assert ((dx[few].double() - want.double()).abs() <= bound).all()


def _magnitude(x, W, dout):
    """A bound of the sum of |dz| |W| for each entry of dx: |act'| <= 1.1, |act| <= |g| (silu)."""
    z = x.double().abs() @ W.double().abs().t()
    F = W.shape[0] // 2
    dz = torch.cat([1.1 * dout.double().abs() * z[:, F:], dout.double().abs() * z[:, :F]], 1)
    return dz @ W.double().abs()


@pytest.mark.parametrize("N,F,dtype", [(256, 2 ** 22 - 64, torch.bfloat16), (128, 2 ** 23 - 64, torch.float32)])
def test_gradients_of_the_longest_rows(N, F, dtype):
    """The rows of a tile of dx reach as far as its offsets do: the tokens in the other order give the same bits."""
    d = 8
    g = torch.Generator(device="cuda").manual_seed(2)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=dtype)   # noqa: E731
    x, W, dout = new(N, d), new(2 * F, d) / F ** 0.5, new(N, F)
    dx, _ = prn.gated_ffn_backward(dout, x, W, want_W=False)
    other, _ = prn.gated_ffn_backward(dout.flip(0), x.flip(0), W, want_W=False)
    assert torch.isfinite(dx).all() and torch.equal(dx, other.flip(0))
    assert len(torch.unique(dx, dim=0)) == N


# fp32 with more than 256 channels and at least 192 tiles of 256 tokens x 128 outputs: the gradients' 256-row tiles,
# 192 columns wide, and (500 and 512 channels) 256
LARGE_FP32 = [(5003, 517, 1387), (6144, 264, 1024), (12289, 260, 513), (3333, 384, 1900), (49157, 257, 33), (6200, 500, 1000),
              (6144, 512, 1024)]


@pytest.mark.parametrize("N,d,F", LARGE_FP32)
def test_large_tiles_of_fp32(N, d, F):
    _check(*_case(N, d, F, torch.float32, seed=d), "silu", torch.float32)


@pytest.mark.parametrize("d", [264, 505])   # 192 columns and 256
def test_what_is_not_finite_on_large_tiles_of_fp32(d):
    N, F = 6151, 1030
    x, W, dout = _case(N, d, F, torch.float32)
    out, (dx, dW) = prn.gated_ffn(x, W), prn.gated_ffn_backward(dout, x, W)
    for bad in (float("nan"), float("inf"), float("-inf")):
        y, g, V = x.clone(), dout.clone(), W.clone()
        y[300, 5] = bad
        out2, (dx2, _) = prn.gated_ffn(y, W), prn.gated_ffn_backward(dout, y, W)
        rest = torch.arange(N, device="cuda") != 300
        assert torch.equal(out2[rest], out[rest]) and torch.equal(dx2[rest], dx[rest])
        assert not torch.isfinite(out2[300]).all() and not torch.isfinite(dx2[300]).all()
        g[6150, 1029] = bad   # the last output of the last token
        dx2, dW2 = prn.gated_ffn_backward(g, x, W)
        assert torch.equal(dx2[:-1], dx[:-1]) and not torch.isfinite(dx2[-1]).any()
        same = torch.ones(2 * F, dtype=torch.bool, device="cuda")
        same[1029] = same[F + 1029] = False
        assert torch.equal(dW2[same], dW[same]) and not torch.isfinite(dW2[~same]).any()
        V[700, 100] = bad   # an output's gate
        out2, (_, dW2) = prn.gated_ffn(x, V), prn.gated_ffn_backward(dout, x, V)
        same[:] = True
        same[700] = same[F + 700] = False
        assert torch.equal(out2[:, same[:F]], out[:, same[:F]]) and torch.equal(dW2[same], dW[same])
