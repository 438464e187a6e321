"""Dropout on the GPU against oracle.gated: the same elements, bit for bit, and
their values to the roundings of a product and a sum in fp32 and the output's."""
import numpy as np
import pytest
import torch

import nonlinear_rnn_amd as prn
from nonlinear_rnn_amd import binding as B
from oracle import gated

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
SEEDS = [(0, 0), (1, 5), ((1 << 63) + 12345, (1 << 40) + 3), (-1, -1)]


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2047, 2048, 2049, 20011])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0, 1.0 / 65536, 65535 / 65536])
def test_elements_and_values(n, p, dtype):
    g = torch.Generator().manual_seed(n)
    x, r = (torch.randn(n, generator=g).to(dtype).cuda() for _ in range(2))
    seed, offset = SEEDS[n % len(SEEDS)]
    m = (1 << 64) - 1
    keep = gated.kept(n, p, seed & m, offset & m)
    ones = prn.dropout(torch.ones_like(x), p, seed=seed, offset=offset)
    assert ((_np(ones) != 0) == keep).all()
    for res in (None, r):
        want = gated.dropout(_np(x), p, seed & m, offset & m, None if res is None else _np(res))
        got = _np(prn.dropout(x, p, seed=seed, offset=offset, residual=res))
        part = np.abs(want - (0.0 if res is None else _np(r)))
        tol = 2 * 2.0 ** -24 * (part + np.abs(want)) * (1 + HALF[dtype]) + HALF[dtype] * np.abs(want)
        assert (np.abs(got - want) <= tol).all()
        if res is not None:
            assert (got[~keep] == _np(r)[~keep]).all()


def test_the_mask_is_the_same_for_every_type_shape_and_direction():
    x = torch.rand(6, 35, 11, device="cuda") + 1.0
    a = prn.dropout(x, 0.3, seed=9, offset=2)
    b = prn.dropout(x.bfloat16().view(-1), 0.3, seed=9, offset=2).view_as(x)
    c = prn.dropout_backward(x.transpose(0, 2).contiguous().transpose(0, 2), 0.3, seed=9, offset=2)
    assert torch.equal(a != 0, b != 0) and torch.equal(a, c)
    for other in (dict(seed=10, offset=2), dict(seed=9, offset=3), dict(seed=9 + (1 << 32), offset=2),
                  dict(seed=9, offset=2 + (1 << 32))):
        assert not torch.equal(prn.dropout(x, 0.3, **other) != 0, a != 0)


@pytest.mark.parametrize("dtype,n", [(torch.float32, (1 << 25) + 13), (torch.bfloat16, (1 << 26) + 5)])
def test_large_tensors(dtype, n):
    """Past 128 MB, against pieces of the same numbers: a piece that starts at a block has the blocks from there on."""
    x, r = torch.randn(n, device="cuda").to(dtype), torch.randn(n, device="cuda").to(dtype)
    out, dx = prn.dropout(x, 0.3, seed=21, offset=4, residual=r), prn.dropout_backward(x, 0.3, seed=21, offset=4)
    small = prn.dropout(x[:1 << 20], 0.3, seed=21, offset=4, residual=r[:1 << 20])
    assert torch.equal(out[:1 << 20], small)
    for lo in (0, 8 * ((n - 3000) // 8)):   # the first and the last blocks, one by one
        hi = min(n, lo + 3000)
        halves = gated.philox(np.arange(lo // 8, (hi + 7) // 8), 4, 21)
        keep = np.stack([halves & 0xFFFF, halves >> 16], -1).reshape(-1)[:hi - lo] >= round(0.3 * 65536)
        assert ((_np(dx[lo:hi]) != 0) == keep).all()
        assert (_np(out[lo:hi])[~keep] == _np(r[lo:hi])[~keep]).all()


def test_what_is_dropped_does_not_count():
    x = torch.full((4000,), float("nan"), device="cuda")
    x[::2] = float("inf")
    r = torch.randn(4000, device="cuda")
    keep = torch.from_numpy(gated.kept(4000, 0.4, 3, 1)).cuda()
    out = prn.dropout(x, 0.4, seed=3, offset=1, residual=r)
    assert torch.equal(out[~keep], r[~keep]) and not torch.isfinite(out[keep]).any()


def test_in_place_through_the_binding():
    x, r = torch.randn(5000, device="cuda"), torch.randn(5000, device="cuda")
    want = prn.dropout(x, 0.2, seed=4, residual=r)
    for out in (x.clone(), r.clone()):
        a, b = (out, r) if torch.equal(out, x) else (x, out)
        B.prn_dropout(a, out, p=0.2, seed=4, residual=b)
        assert torch.equal(out, want)


def test_a_seed_on_the_device():
    x = torch.randn(3000, device="cuda")
    state = torch.tensor([11, 0], device="cuda")
    graph = torch.cuda.CUDAGraph()
    prn.dropout(x, 0.5, seed=state)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = prn.dropout(x, 0.5, seed=state)
    for k in range(4):
        state[1] = k
        want = prn.dropout(x, 0.5, seed=11, offset=k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), k


def test_autograd():
    x, r = (torch.randn(40, 33, device="cuda", requires_grad=True) for _ in range(2))
    w = torch.randn(40, 33, device="cuda")
    state = torch.tensor([5, 6], device="cuda")
    for kw in (dict(seed=5, offset=6), dict(seed=state)):
        state[0], state[1] = 5, 6
        y = prn.dropout_apply(x, 0.25, residual=r, **kw)
        state[1] = 99   # the backward pass is of the call as it was
        dx, dr = torch.autograd.grad((y * w).sum(), (x, r))
        assert torch.equal(dx, prn.dropout(w, 0.25, seed=5, offset=6)) and torch.equal(dr, w)
    g, = torch.autograd.grad(prn.dropout_apply(x, 0.5, seed=1).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        g.square().sum().backward()


def test_nothing_and_refusals():
    x = torch.zeros(4, 8, device="cuda")
    assert prn.dropout(x[:0], 0.5, seed=1).shape == (0, 8)
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(B.PrnError):
            prn.dropout(x, p, seed=1)
    with pytest.raises(ValueError):
        prn.dropout(x, 0.5, seed=1, residual=torch.zeros(8, 4, device="cuda"))
    with pytest.raises(TypeError):
        prn.dropout(x, 0.5, seed=1, residual=x.bfloat16())
    with pytest.raises(TypeError):
        prn.dropout(x.half(), 0.5, seed=1)
    with pytest.raises(TypeError):
        prn.dropout(x, 0.5, seed=torch.tensor([1, 2], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        prn.dropout(x, 0.5, seed=torch.tensor([1, 2], device="cuda"), offset=1)


def test_offsets_past_32_bits():
    """2^32 + 12345 elements: the last ones' numbers are those of their own index."""
    n = 2 ** 32 + 12345
    out = prn.dropout(torch.ones(n, dtype=torch.bfloat16, device="cuda"), 0.25, seed=11, offset=3)
    for at in (2 ** 31, 2 ** 32, n - n % 8 - 64):
        words = gated.philox(np.arange(at // 8, at // 8 + 8, dtype=np.int64), 3, 11)
        keep = np.stack([words & 0xFFFF, words >> 16], -1).reshape(-1) >= round(0.25 * 65536)
        assert np.array_equal(out[at:at + 64].float().cpu().numpy() != 0, keep)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 8, 13, 5003, 1 << 20, (1 << 26) + 5])
def test_in_place_over_every_operand(n, dtype):
    """The result over x, over the residual, and over a tensor that is both, for each launch there is."""
    g = torch.Generator(device="cuda").manual_seed(n)
    x, r = (torch.randn(n, generator=g, device="cuda").to(dtype) for _ in range(2))
    want, alone, both = (prn.dropout(x, 0.3, seed=6, residual=q) for q in (r, None, x))
    out = x.clone()
    B.prn_dropout(out, out, p=0.3, seed=6, residual=r)
    assert torch.equal(out, want)
    out.copy_(r)
    B.prn_dropout(x, out, p=0.3, seed=6, residual=out)
    assert torch.equal(out, want)
    out.copy_(x)
    B.prn_dropout(out, out, p=0.3, seed=6)
    assert torch.equal(out, alone)
    out.copy_(x)
    B.prn_dropout(out, out, p=0.3, seed=6, residual=out)
    assert torch.equal(out, both)
