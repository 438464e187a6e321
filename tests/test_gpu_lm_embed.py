"""GPU parity of the embedding lookup and its gradient against oracle.lm.

Bands, per element, u = half a step of the storage type (torch.finfo.eps / 2):
  lookup    u |ref|, plus 2^-24 |ref| for the fp32 product before a bf16 rounding
  gradient  u |ref| + (c + 2) 2^-24 sum |scale dout| for c summed rows (c - 1
            fp32 additions, the scale's product, and their second orders)
"""
import numpy as np
import pytest
import torch

import nonlinear_rnn_amd as prn
from gpu_helpers import TORCH_DT, say, to_f64
from nonlinear_rnn_amd import binding as B
from oracle import lm as olm

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24


def _u(dtype):
    return torch.finfo(TORCH_DT[dtype]).eps / 2


def _draw(kind, N, V, rng):
    if kind == "uniform":
        return rng.integers(0, V, N)
    if kind == "same":
        return np.full(N, V // 2)
    if kind == "skewed":
        return np.minimum((V ** rng.random(N)).astype(np.int64) - 1, V - 1).clip(0)
    if kind == "many":   # run lengths around the cuts of a very frequent token's chunks
        lengths = [511, 512, 513, 527, 528, 529, 1023, 1024, 1025, 1040, 2049]
        return rng.permutation(np.concatenate([np.repeat(np.arange(len(lengths)), lengths), rng.integers(20, V, N)])[:N])
    # "runs": run lengths around the cut of a frequent token's rows, then shuffled
    lengths = [1, 2, 15, 16, 17, 62, 63, 64, 65, 66, 127, 128, 129, 191, 192, 193, 300]
    ids = np.repeat(np.arange(len(lengths)), lengths)[:N]
    ids = np.concatenate([ids, np.full(N - len(ids), V - 1)])
    return rng.permutation(ids % V)


def _check(N, V, d, dtype, kind, ids=np.int64, scale=1.5, pad=None, odd=False):
    say(f"[case] embed N={N} V={V} d={d} {dtype} {kind} {ids.__name__} pad={pad}")
    rng = np.random.default_rng(N + V + d)
    tok = _draw(kind, N, V, rng)
    if odd:
        tok[::7] = -3
        tok[1::11] = V
        tok[2::13] = 2 ** 31 - 1
    table = torch.from_numpy(rng.standard_normal((V, d))).to(TORCH_DT[dtype])
    dout = torch.from_numpy(rng.standard_normal((N, d))).to(TORCH_DT[dtype])
    dev = torch.from_numpy(tok.astype(ids)).cuda()
    out = prn.embed(dev, table.cuda(), scale=scale, pad_id=pad)
    ref = olm.embed(tok, to_f64(table), scale, pad)
    got = to_f64(out)
    assert (np.isnan(got) == np.isnan(ref)).all()
    ok = ~np.isnan(ref)
    assert (np.abs(got - ref)[ok] <= ((_u(dtype) + 2 * E24) * np.abs(ref))[ok]).all()
    grad = prn.embed_backward(dout.cuda(), dev, V, scale=scale, pad_id=pad)
    ref, size, count = olm.embed_backward(to_f64(dout), tok, V, scale, pad)
    err = np.abs(to_f64(grad) - ref)
    assert (err <= _u(dtype) * np.abs(ref) + (count[:, None] + 2) * E24 * size).all(), float(err.max())
    again = prn.embed_backward(dout.cuda(), dev, V, scale=scale, pad_id=pad)
    assert torch.equal(grad, again)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,d,kind", [
    (1, 1, 1, "uniform"), (1, 9, 8, "uniform"), (16, 5, 3, "uniform"), (17, 300, 7, "skewed"), (63, 2, 16, "same"),
    (64, 2, 16, "same"), (65, 2, 20, "same"), (129, 40, 12, "same"), (1100, 64, 24, "runs"), (2000, 50, 40, "runs"),
    (2047, 512, 64, "uniform"), (2048, 511, 130, "skewed"), (2049, 513, 512, "skewed"), (5000, 300, 1000, "uniform"),
    (9000, 131075, 8, "skewed"), (4100, 300000, 16, "uniform"), (5000, 1000, 256, "same"), (20000, 700, 33, "skewed"),
])
def test_embed_matches_oracle(N, V, d, kind, dtype):
    _check(N, V, d, dtype, kind)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,d,kind", [
    (8191, 700, 12, "skewed"), (8192, 9000, 8, "uniform"), (8193, 9000, 8, "uniform"),   # both sorts
    (8192, 524287, 4, "uniform"), (8192, 524288, 4, "uniform"),                           # a word for key and position, or not
    (8190, 60, 24, "many"), (12000, 3000, 260, "many"),
])
def test_embed_gradient_at_the_cuts(N, V, d, kind, dtype):
    _check(N, V, d, dtype, kind)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ids", [np.int32, np.int64])
def test_embed_pad_and_tokens_outside_the_table(dtype, ids):
    _check(3000, 90, 48, dtype, "skewed", ids, pad=0, odd=True)
    _check(700, 90, 48, dtype, "uniform", ids, pad=-3, odd=True)    # a pad id that is no row
    _check(700, 90, 48, dtype, "same", ids, pad=45)                 # nothing but padding


def test_embed_empty_strided_and_misaligned():
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randn(50, 36, generator=g, device="cuda").bfloat16()
    assert prn.embed(torch.empty(0, dtype=torch.int64, device="cuda"), table).shape == (0, 36)
    z = prn.embed_backward(torch.empty(0, 36, device="cuda").bfloat16(),
                           torch.empty(0, dtype=torch.int64, device="cuda"), 50)
    assert z.shape == (50, 36) and not z.any()
    tok = torch.randint(0, 50, (6, 10), generator=g, device="cuda")
    want = prn.embed(tok, table)
    assert want.shape == (6, 10, 36)
    assert torch.equal(prn.embed(tok.t(), table), want.transpose(0, 1))                      # strided tokens
    wide = torch.randn(50, 40, generator=g, device="cuda").bfloat16()
    assert torch.equal(prn.embed(tok, wide[:, 1:37]), prn.embed(tok, wide[:, 1:37].contiguous()))
    flat = torch.empty(50 * 36 + 1, dtype=torch.bfloat16, device="cuda")
    flat[1:] = table.view(-1)
    assert torch.equal(prn.embed(tok, flat[1:].view(50, 36)), want)                          # 2-byte aligned table
    dout = torch.randn(10, 6, 36, generator=g, device="cuda").bfloat16().transpose(0, 1)
    assert torch.equal(prn.embed_backward(dout, tok, 50), prn.embed_backward(dout.contiguous(), tok, 50))
    dflat = torch.empty(60 * 36 + 1, dtype=torch.bfloat16, device="cuda")
    dflat[1:] = dout.reshape(-1)
    assert torch.equal(prn.embed_backward(dflat[1:].view(6, 10, 36), tok, 50),
                       prn.embed_backward(dout.contiguous(), tok, 50))


def test_embed_autograd_against_the_formula():
    g = torch.Generator(device="cuda").manual_seed(2)
    table = torch.randn(30, 20, generator=g, device="cuda").requires_grad_()
    tok = torch.randint(0, 30, (4, 50), generator=g, device="cuda")
    w = torch.randn(4, 50, 20, generator=g, device="cuda")
    (prn.embed_apply(tok, table, scale=2.0, pad_id=3) * w).sum().backward()
    assert torch.equal(table.grad, prn.embed_backward(w, tok, 30, scale=2.0, pad_id=3))


def test_embed_on_another_stream_and_in_a_graph():
    g = torch.Generator(device="cuda").manual_seed(3)
    V, d, N = 500, 64, 3000
    table = torch.randn(V, d, generator=g, device="cuda")
    tok = torch.randint(0, 40, (N,), generator=g, device="cuda")
    dout = torch.randn(N, d, generator=g, device="cuda")
    want = prn.embed(tok, table), prn.embed_backward(dout, tok, V)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = prn.embed(tok, table), prn.embed_backward(dout, tok, V)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, grad = prn.embed(tok, table), prn.embed_backward(dout, tok, V)
    for k in range(3):
        tok.copy_(torch.randint(0, 40 + 100 * k, (N,), generator=g, device="cuda"))
        dout.normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, prn.embed(tok, table)) and torch.equal(grad, prn.embed_backward(dout, tok, V))


def test_binding_checks_shapes_and_types():
    tok = torch.zeros(4, dtype=torch.int64, device="cuda")
    table, out = torch.zeros(5, 8, device="cuda"), torch.zeros(4, 8, device="cuda")
    with pytest.raises(TypeError):
        B.prn_embed(tok.to(torch.int16), table, out)
    with pytest.raises(TypeError):
        B.prn_embed(tok, table.half(), out.half())
    with pytest.raises(TypeError):
        B.prn_embed(tok, table, out.bfloat16())
    with pytest.raises(ValueError):
        B.prn_embed(tok, table, out[:3])
    with pytest.raises(ValueError):
        B.prn_embed(tok, table, out.t().contiguous().t())
    with pytest.raises(B.PrnError, match="workspace"):
        B.prn_embed_backward(tok, out, table)


def test_more_tokens_than_one_row_of_a_grid():
    """2^30 tokens and a few, one channel: more threads than one dimension of a launch may have."""
    table = torch.randn(5, 1, device="cuda").bfloat16()
    tok = torch.arange(5, device="cuda", dtype=torch.int32).repeat((1 << 30) // 5 + 2)[:(1 << 30) + 3]
    out = prn.embed(tok, table)
    n = out.shape[0] // 5
    assert torch.equal(out[:5 * n].view(n, 5), table[:, 0].expand(n, 5)) and torch.equal(out[5 * n:], table[:len(out) - 5 * n])


@pytest.mark.parametrize("dtype,N,V,d,kind", [("f32", 640 * 2048, 70000, 2, "skewed"), ("f32", 640 * 2048 + 1, 3000, 2, "uniform"),
                                             ("bf16", 1400007, 300000, 3, "skewed"), ("f32", 2097153, 500, 1, "uniform")])
def test_embed_gradient_of_many_tiles(dtype, N, V, d, kind):
    """640 tiles of 2048 tokens, and more of them, whose counts are summed up in groups of 256 before the scatter."""
    _check(N, V, d, dtype, kind)


def test_embed_gradient_of_a_billion_tokens():
    """2^30 tokens and a few, each 1024 times, one channel: sums of ones are exact.  (Adding up the counts of all
    tiles in every tile would read 600 TB.)"""
    V, n = 1 << 20, (1 << 30) + 5
    tok = torch.arange(n, device="cuda", dtype=torch.int32).bitwise_and_(V - 1)
    grad = prn.embed_backward(torch.ones(n, 1, device="cuda", dtype=torch.bfloat16), tok, V)
    want = torch.full((V, 1), 1024.0, device="cuda")
    want[:5] += 1
    assert torch.equal(grad, want.bfloat16())


def test_the_value_that_stands_for_no_pad_id_is_no_pad_id():
    tok = torch.tensor([-2 ** 63, 1], device="cuda")
    out = prn.embed(tok, torch.ones(4, 24, device="cuda"))
    assert out[0].isnan().all() and (out[1] == 1).all()
