"""The gated linear recurrence on the GPU against oracle.gated in float64.

Tolerances are the oracle's elementwise bounds (gated_scan_bounds, in units of
2^-24) and the output's own rounding, half a step of its storage type; the
gradient of bf16 data starts every chunk from a stored state, half a step off.
"""
import numpy as np
import pytest
import torch

import nonlinear_rnn_amd as prn
from nonlinear_rnn_amd import binding as B
from oracle import gated

pytestmark = pytest.mark.gpu

G = {"glr": 2, "glri": 3}
U24 = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = 1e-30   # below it fp32 loses bits, or all


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _case(cell, Bn, T, d, dtype, cu=None, h0=True, seed=0, spread=8.0):
    g = torch.Generator().manual_seed(seed)
    rows = Bn if cu is None else len(cu) - 1
    new = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()   # noqa: E731
    x = torch.randn(Bn, T, G[cell], d, generator=g)
    x[:, :, 0] += torch.linspace(-2.0, spread, d)
    c = dict(x=x.to(dtype).cuda(), h0=new(rows, 1, d) if h0 else None, dH=new(Bn, T, d),
             dlast=new(rows, 1, d) if h0 else None, cu=None)
    if cu is not None:
        c["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    return c


def _close(name, got, want, bound, dtype):
    got = _np(got)
    tol = bound * U24 * (1 + HALF[dtype]) + HALF[dtype] * np.abs(want) + TINY
    bad = ~(np.abs(got - want) <= tol)
    worst = (np.abs(got - want) / tol).max() if got.size else 0.0
    print(f"  {name}: worst {worst:.3f} of its tolerance", flush=True)
    assert not bad.any(), (name, np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])


def _check(cell, c, dtype, backward=True):
    cu = None if c["cu"] is None else c["cu"].cpu().numpy()
    kw = dict(cell=cell, h0=c["h0"], cu_seqlens=c["cu"])
    H, last = prn.gated_scan(c["x"], return_state=True, **kw)
    x, h0 = _np(c["x"]), _np(c["h0"])
    want_H, want_last = gated.gated_scan(cell, x, h0, cu)
    bounds = gated.gated_scan_bounds(cell, x, h0, cu, _np(c["dH"]), _np(c["dlast"]),
                                     start=HALF[dtype] / U24 if dtype == torch.bfloat16 else 1.0)
    _close("H", H, want_H, bounds["H"], dtype)
    _close("last", last, want_last, bounds["last"], dtype)
    if not backward:
        return H, last
    dx, dh0 = prn.gated_scan_backward(c["dH"], c["x"], H, dstate=c["dlast"], **kw)
    want_dx, want_dh0 = gated.gated_scan_backward(cell, x, _np(c["dH"]), h0, cu, _np(c["dlast"]))
    _close("dxproj", dx, want_dx, bounds["dxproj"], dtype)
    if c["h0"] is None:
        assert dh0 is None
    else:
        _close("dh0", dh0, want_dh0, bounds["dh0"], dtype)
    return H, last, dx, dh0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cell", ["glr", "glri"])
@pytest.mark.parametrize("Bn,T,d", [(1, 1, 1), (3, 1, 130), (2, 2, 64), (1, 7, 63), (2, 8, 65), (1, 63, 2), (2, 64, 5),
                                    (1, 65, 128), (3, 127, 33), (2, 129, 250), (1, 1000, 3), (1, 4100, 64), (5, 700, 1)])
def test_rectangular(cell, Bn, T, d, dtype):
    _check(cell, _case(cell, Bn, T, d, dtype, h0=T % 2 == 0), dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cell", ["glr", "glri"])
@pytest.mark.parametrize("cu", [[0, 1], [0, 0, 5, 5, 5, 9, 9], [0, 64, 128, 129, 200], [0, 63, 63, 64, 65, 300],
                                list(range(0, 90)), [0, 2, 2000, 2001, 4000]])
@pytest.mark.parametrize("h0", [False, True])
def test_ragged(cell, cu, h0, dtype):
    _check(cell, _case(cell, 1, cu[-1], 70, dtype, cu, h0=h0, seed=len(cu)), dtype)


@pytest.mark.parametrize("cell", ["glr", "glri"])
def test_many_sequences(cell):
    rng = np.random.default_rng(3)
    cu = [0, *sorted(rng.integers(0, 3001, 400).tolist()), 3000]
    cu = sorted(min(v, 3000) for v in cu)
    _check(cell, _case(cell, 1, 3000, 20, torch.float32, cu), torch.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cell", ["glr", "glri"])
@pytest.mark.parametrize("Bn,T,d", [(300, 150, 20), (130, 70, 260), (260, 1, 64), (256, 129, 64), (3, 256, 40), (3, 257, 40),
                                    (1, 2049, 7), (2, 513, 128)])
def test_on_either_side_of_a_limit(cell, Bn, T, d, dtype):
    """Chains enough for a workgroup each, or not, and lengths about the chunks of both ways."""
    _check(cell, _case(cell, Bn, T, d, dtype, h0=Bn % 2 == 0, seed=T), dtype)


@pytest.mark.parametrize("cu", [None, [0, 0, 321, 9000, 17003]])
@pytest.mark.parametrize("cell,d,dtype", [("glr", 250, torch.float32), ("glri", 250, torch.float32), ("glri", 251, torch.bfloat16)])
def test_chunks_by_rounds(cell, d, dtype, cu):
    """More chunks than a round of the device has, and longer ones in one round less."""
    _check(cell, _case(cell, 1, 17003, d, dtype, cu), dtype)


def test_a_long_chain():
    """Hundreds of chunks of one chain: the look-back over more than 64 of them."""
    for cell, dtype in (("glr", torch.float32), ("glri", torch.bfloat16)):
        c = _case(cell, 1, 60000, 3, dtype)
        _check(cell, c, dtype)


def test_a_wait_that_gives_up(monkeypatch):
    """PRN_SPIN_LIMIT=0: every wait gives up at once.  The kernel ends, the error word is set, what has no wait
    before it is right and the rest NaN; without the limit the same call is right again and the word stays."""
    c = _case("glr", 1, 3000, 64, torch.float32)
    H, err = torch.empty(1, 3000, 64, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    n = max(f("glr", torch.float32, 1, 3000, 64) for f in (B.prn_gated_scan_workspace_bytes,
                                                           B.prn_gated_scan_backward_workspace_bytes))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    want = prn.gated_scan(c["x"], cell="glr", h0=c["h0"])
    want_dx, _ = prn.gated_scan_backward(c["dH"], c["x"], want, cell="glr", h0=c["h0"])
    dx = torch.empty_like(c["x"])
    kw = dict(cell="glr", h0=c["h0"], workspace=ws, error_out=err)
    monkeypatch.setenv("PRN_SPIN_LIMIT", "0")
    B.prn_gated_scan(c["x"], H, **kw)
    assert err.item() == B.PRN_FAULT_LOOKBACK
    assert torch.equal(H[0, :256], want[0, :256]) and torch.isnan(H[0, 256:]).all()
    err.zero_()
    B.prn_gated_scan_backward(c["x"], want, c["dH"], dx, **kw)
    assert err.item() == B.PRN_FAULT_LOOKBACK
    last = 3000 // 128 * 128   # the last chunk's first step
    assert torch.equal(dx[0, last:], want_dx[0, last:]) and torch.isnan(dx[0, :last]).all()
    monkeypatch.delenv("PRN_SPIN_LIMIT")
    B.prn_gated_scan(c["x"], H, **kw)
    B.prn_gated_scan_backward(c["x"], H, c["dH"], dx, **kw)
    assert torch.equal(H, want) and torch.equal(dx, want_dx) and err.item() == B.PRN_FAULT_LOOKBACK


def test_no_step_and_no_row():
    """T = 0: the final state is the initial one, its gradient passes through."""
    for cu in (None, [0, 0, 0]):
        rows = 2
        Bn = 2 if cu is None else 1
        x = torch.empty(Bn, 0, 2, 6, device="cuda")
        h0 = torch.randn(rows, 1, 6, device="cuda")
        c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
        H, last = prn.gated_scan(x, cell="glr", h0=h0, cu_seqlens=c, return_state=True)
        assert H.shape == (Bn, 0, 6) and torch.equal(last, h0)
        dx, dh0 = prn.gated_scan_backward(H, x, H, cell="glr", h0=h0, cu_seqlens=c, dstate=2 * h0)
        assert dx.shape == x.shape and torch.equal(dh0, 2 * h0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [200, 5000])
def test_one_sequence_is_not_anothers(T, dtype):
    """NaN and infinities of a sequence stay there, whatever the ranges and chunks; the others keep their bits."""
    cu = [0, 3, T // 2 + 1, T // 2 + 40, T]
    for cell in ("glr", "glri"):
        c = _case(cell, 1, T, 40, dtype, cu, seed=4)
        kw = dict(cell=cell, cu_seqlens=c["cu"])
        H, last = prn.gated_scan(c["x"], h0=c["h0"], return_state=True, **kw)
        dx, dh0 = prn.gated_scan_backward(c["dH"], c["x"], H, h0=c["h0"], dstate=c["dlast"], **kw)
        for j in range(4):
            lo, hi = cu[j], cu[j + 1]
            for bad in (float("nan"), float("inf"), float("-inf")):
                x, h0, dH, dlast = c["x"].clone(), c["h0"].clone(), c["dH"].clone(), c["dlast"].clone()
                x[0, lo:hi], h0[j], dH[0, lo:hi], dlast[j] = bad, bad, bad, bad
                H2, last2 = prn.gated_scan(x, h0=h0, return_state=True, **kw)
                dx2, dh2 = prn.gated_scan_backward(dH, x, H2, h0=h0, dstate=dlast, **kw)
                keep = torch.ones(T, dtype=torch.bool, device="cuda")
                keep[lo:hi] = False
                rest = [k for k in range(4) if k != j]
                assert torch.equal(H2[0, keep], H[0, keep]) and torch.equal(last2[rest], last[rest])
                assert torch.equal(dx2[0, keep], dx[0, keep]) and torch.equal(dh2[rest], dh0[rest])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cell", ["glr", "glri"])
@pytest.mark.parametrize("cu,T", [([0, 3, 90], 250), ([0, 5, 5, 300, 700], 1000), ([0, 0, 512], 2000), ([0, 0], 300), ([0, 0], 30)])
def test_steps_behind_the_last_sequence(cu, T, cell, dtype):
    """A pack of a fixed size that ends early: the sequences' results to the bit, zeros behind, whatever is there."""
    c, n = _case(cell, 1, T, 40, dtype, cu), cu[-1]
    for t in (c["x"], c["dH"]):
        t[:, n:] = float("nan")
    kw = dict(cell=cell, h0=c["h0"], cu_seqlens=c["cu"])
    H, last = prn.gated_scan(c["x"], return_state=True, **kw)
    dx, dh0 = prn.gated_scan_backward(c["dH"], c["x"], H, dstate=c["dlast"], **kw)
    x, dH = (t[:, :n].contiguous() for t in (c["x"], c["dH"]))
    want_H, want_last = prn.gated_scan(x, return_state=True, **kw)
    want_dx, want_dh0 = prn.gated_scan_backward(dH, x, want_H, dstate=c["dlast"], **kw)
    assert torch.equal(H[:, :n], want_H) and torch.equal(last, want_last)
    assert torch.equal(dx[:, :n], want_dx) and torch.equal(dh0, want_dh0)
    assert (H[:, n:] == 0).all() and (dx[:, n:] == 0).all()


def test_a_nan_reaches_all_that_comes_after_it():
    c = _case("glr", 1, 4000, 64, torch.float32, h0=False)
    c["x"][0, 100, 1, 7] = float("nan")
    H, last = prn.gated_scan(c["x"], cell="glr", return_state=True)
    assert torch.isnan(H[0, 100:, 7]).all() and torch.isnan(last[0, 0, 7])
    assert not torch.isnan(H[0, :100]).any() and not torch.isnan(H[0, :, :7]).any() and not torch.isnan(H[0, :, 8:]).any()


def test_held_and_open_gates_are_exact():
    """x_f = inf keeps the state, -inf replaces it, without NaN; the lowest finite value acts as -inf."""
    T = 3000
    x = torch.zeros(1, T, 2, 5, device="cuda")
    x[:, :, 0] = float("inf")
    x[:, :, 1] = torch.randn(1, T, 5, device="cuda")
    x[0, 1000, 0], x[0, 2500, 0] = float("-inf"), torch.finfo(torch.float32).min
    h0 = torch.randn(1, 1, 5, device="cuda")
    H, last = prn.gated_scan(x, cell="glr", h0=h0, return_state=True)
    want = torch.cat([h0[0].expand(1000, 5), x[0, 1000, 1].expand(1500, 5), x[0, 2500, 1].expand(500, 5)])
    assert torch.equal(H[0], want) and torch.equal(last[0, 0], want[-1])
    dx, dh0 = prn.gated_scan_backward(torch.ones_like(H), x, H, cell="glr", h0=h0)
    assert torch.equal(dh0, torch.full_like(h0, 1000.0)) and (dx[:, :, 0] == 0).all()
    assert torch.equal(dx[0, :, 1], torch.where((x[0, :, 0] < 0), torch.tensor([1500.0, 500.0], device="cuda").repeat_interleave(
        torch.tensor([2000, 1000], device="cuda"))[:, None], torch.zeros(5, device="cuda")))


def test_long_memory_keeps_its_precision():
    """Gates of 1 - 2^-11: the state is a sum over thousands of steps."""
    c = _case("glr", 1, 20000, 64, torch.float32, h0=True, spread=8.0)
    _check("glr", c, torch.float32)


@pytest.mark.parametrize("cell", ["glr", "glri"])
def test_twice_the_same_bits_and_other_layouts(cell):
    c = _case(cell, 2, 3001, 48, torch.bfloat16)
    kw = dict(cell=cell, h0=c["h0"])
    H, last = prn.gated_scan(c["x"], return_state=True, **kw)
    dx, dh0 = prn.gated_scan_backward(c["dH"], c["x"], H, dstate=c["dlast"], **kw)
    for _ in range(3):
        H2, last2 = prn.gated_scan(c["x"], return_state=True, **kw)
        assert torch.equal(H, H2) and torch.equal(last, last2)
    # strided and unaligned views
    wide = torch.empty(2, 3001, G[cell], 49, dtype=torch.bfloat16, device="cuda")
    wide[..., 1:] = c["x"]
    odd = torch.empty(dH_n := c["dH"].numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view_as(c["dH"])
    odd.copy_(c["dH"])
    assert dH_n and odd.data_ptr() % 16
    H2, last2 = prn.gated_scan(wide[..., 1:], return_state=True, **kw)
    dx2, dh2 = prn.gated_scan_backward(odd, wide[..., 1:], H2, dstate=c["dlast"], **kw)
    assert torch.equal(H, H2) and torch.equal(last, last2) and torch.equal(dx, dx2) and torch.equal(dh0, dh2)


def test_rows_do_not_depend_on_the_others():
    """A row of a batch against the row alone, within twice the bound (another cut of time sums in another order)."""
    c = _case("glri", 6, 900, 96, torch.float32)
    H = prn.gated_scan(c["x"], cell="glri", h0=c["h0"])
    x, h0 = _np(c["x"]), _np(c["h0"])
    tol = 2 * gated.gated_scan_bounds("glri", x, h0)["H"] * U24 + 2 * U24 * np.abs(_np(H)) + TINY
    for b in range(6):
        alone = prn.gated_scan(c["x"][b:b + 1], cell="glri", h0=c["h0"][b:b + 1])
        assert (np.abs(_np(alone)[0] - _np(H)[b]) <= tol[b]).all()


@pytest.mark.parametrize("ragged", [False, True])
def test_autograd(ragged):
    cu = [0, 40, 40, 150] if ragged else None
    c = _case("glr", 1 if ragged else 3, 150, 24, torch.float32, cu)
    x, h0 = c["x"].requires_grad_(), c["h0"].requires_grad_()
    H, last = prn.gated_scan_apply(x, cell="glr", h0=h0, cu_seqlens=cu, return_state=True)
    dx, dh0 = torch.autograd.grad((H * c["dH"]).sum() + (last * c["dlast"]).sum(), (x, h0))
    want = prn.gated_scan_backward(c["dH"], x, H, cell="glr", h0=h0, cu_seqlens=c["cu"], dstate=c["dlast"])
    assert torch.equal(dx, want[0]) and torch.equal(dh0, want[1])
    # either output alone, and no initial state
    last_only, = torch.autograd.grad(prn.gated_scan_apply(x, cell="glr", h0=h0, cu_seqlens=cu, return_state=True)[1].sum(), x)
    want = prn.gated_scan_backward(torch.zeros_like(H), x, H, cell="glr", h0=h0, cu_seqlens=c["cu"],
                                   dstate=torch.ones_like(h0))[0]
    assert torch.equal(last_only, want)
    H, = (prn.gated_scan_apply(x, cell="glr", cu_seqlens=cu),)
    g, = torch.autograd.grad(H.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        g.square().sum().backward()


@pytest.mark.parametrize("T", [1, 300, 3000])
def test_captured_and_replayed(T):
    """Forward and backward in a graph, new inputs between replays, eager work beside it."""
    c = _case("glri", 2, T, 64, torch.float32)
    x, dH = c["x"].clone(), c["dH"].clone()

    def both():
        H, last = prn.gated_scan(x, cell="glri", h0=c["h0"], return_state=True)
        return H, last, *prn.gated_scan_backward(dH, x, H, cell="glri", h0=c["h0"], dstate=c["dlast"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for k in range(4):
        new = _case("glri", 2, T, 64, torch.float32, seed=10 + k)
        x.copy_(new["x"])
        dH.copy_(new["dH"])
        want = [t.clone() for t in both()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), k


def test_two_streams_at_once():
    c = [_case("glr", 2, 2500, 64, torch.float32, seed=s) for s in (1, 2)]
    want = [prn.gated_scan(k["x"], cell="glr", h0=k["h0"]) for k in c]
    streams = [torch.cuda.Stream() for _ in c]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(prn.gated_scan(c[i]["x"], cell="glr", h0=c[i]["h0"]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in (0, 1) for g in got[i])


# ------------------------------------------------------------------ projection and serving step ---

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cell", ["glr", "glri"])
@pytest.mark.parametrize("slots,d_in,d", [(1, 1, 1), (3, 16, 40), (16, 100, 33), (17, 513, 64), (64, 512, 130), (200, 70, 17)])
def test_decode_step(cell, slots, d_in, d, dtype):
    """Projection and step in one launch, without rounding in between: z is a sum of d_in products, off by
    (d_in + 2) 2^-24 of their magnitudes."""
    g = torch.Generator().manual_seed(slots)
    new = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    x, W = new(slots, d_in).to(dtype).cuda(), (new(G[cell] * d, d_in) / d_in ** 0.5).to(dtype).cuda()
    bias, h = new(G[cell] * d).cuda(), new(slots, 1, d).to(dtype).cuda()
    for b, s in ((bias, h), (None, None)):
        out, flat = torch.empty_like(h), torch.empty(slots, d, dtype=dtype, device="cuda")
        B.prn_decode_step(x, W, b, None, out, cell=cell, state_in=s, h_out=flat)
        assert torch.equal(out[:, 0], flat)
        z = _np(x) @ _np(W).T + (0.0 if b is None else _np(b))
        ez = (d_in + 2) * (np.abs(_np(x)) @ np.abs(_np(W)).T + (0.0 if b is None else np.abs(_np(b))))
        z, ez = z.reshape(slots, 1, G[cell], d), ez.reshape(slots, 1, G[cell], d)
        h0 = np.zeros((slots, 1, d)) if s is None else _np(s)
        want = gated.gated_scan(cell, z, h0)[1]
        bound = gated.gated_scan_bounds(cell, z, h0)["last"]
        # |s'| <= 1/4 and |s| <= 1; the products of two errors are below 2^-24 of the rest
        v, ev = np.abs(z[:, :, -1]), ez[:, :, -1]
        i = np.ones_like(v)
        moved = 0.25 * ez[:, :, 0] * (np.abs(h0) + (v if cell == "glr" else 0.0)) + i * ev
        if cell == "glri":
            moved += 0.25 * ez[:, :, 1] * v
        _close("state", out, want, bound + 1.01 * moved, dtype)


@pytest.mark.parametrize("cell", ["glr", "glri"])
def test_projection_scan_and_steps_agree(cell):
    """A prompt through the projection and the scan, then single steps on its carry, against the whole sequence."""
    g = torch.Generator().manual_seed(5)
    Bn, T, d_in, d = 3, 90, 64, 48
    new = lambda *s: torch.randn(*s, generator=g).cuda()   # noqa: E731
    x, W, bias = new(Bn, T, d_in), new(G[cell] * d, d_in) / 8, new(G[cell] * d)
    H, last = prn.gated_scan(prn.input_proj(x, W, bias, cell=cell), cell=cell, return_state=True)
    _, carry = prn.gated_scan(prn.input_proj(x[:, :60], W, bias, cell=cell), cell=cell, return_state=True)
    for t in range(60, T):
        new_carry = torch.empty_like(carry)
        B.prn_decode_step(x[:, t].contiguous(), W, bias, None, new_carry, cell=cell, state_in=carry)
        carry = new_carry
        # both are within a few 1e-6 of the truth (sums of 64 products of order one, gates below 1): 24 x 64 x 2^-24
        assert (carry[:, 0] - H[:, t]).abs().max().item() <= 1e-4
    assert torch.equal(H[:, -1], last[:, 0])


@pytest.mark.parametrize("cell", ["glr", "glri"])
def test_projection_gradients(cell):
    g = torch.Generator().manual_seed(6)
    new = lambda *s: torch.randn(*s, generator=g).cuda()   # noqa: E731
    x, W, bias = new(2, 50, 32).requires_grad_(), (new(G[cell] * 24, 32) / 6).requires_grad_(), new(G[cell] * 24).requires_grad_()
    dH = new(2, 50, 24)
    H = prn.gated_scan_apply(prn.input_proj_apply(x, W, bias, cell=cell), cell=cell)
    grads = torch.autograd.grad((H * dH).sum(), (x, W, bias))
    xd, Wd, bd = _np(x), _np(W), _np(bias)
    z = (xd @ Wd.T + bd).reshape(2, 50, G[cell], 24)
    dz = gated.gated_scan_backward(cell, z, _np(dH))[0].reshape(100, -1)
    for got, want in zip(grads, (dz @ Wd, dz.T @ xd.reshape(100, -1), dz.sum(0))):
        err = np.abs(_np(got).reshape(want.shape) - want).max() / np.abs(want).max()
        assert err <= 2e-5, err   # a hundred products, each factor off by some 1e-6 at most, relative to the largest


def test_refusals():
    x = torch.zeros(2, 4, 2, 8, device="cuda")
    H = torch.zeros(2, 4, 8, device="cuda")
    pack = torch.zeros(1, 6, 2, 8, device="cuda")
    for bad in ([0], [], [[0, 6]]):
        with pytest.raises(ValueError):
            prn.gated_scan(pack, cell="glr", cu_seqlens=torch.tensor(bad, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        prn.gated_scan(x, cell="gru")
    with pytest.raises(ValueError):
        prn.gated_scan(x, cell="glri")
    with pytest.raises(ValueError):
        prn.gated_scan(x[0], cell="glr")
    with pytest.raises(ValueError):
        prn.gated_scan(x, cell="glr", h0=torch.zeros(2, 8, device="cuda"))
    with pytest.raises(TypeError):
        prn.gated_scan(x, cell="glr", h0=torch.zeros(2, 1, 8, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        prn.gated_scan(x.half(), cell="glr")
    with pytest.raises(B.PrnError):   # a pack has one row
        prn.gated_scan(x, cell="glr", cu_seqlens=torch.tensor([0, 4], dtype=torch.int32, device="cuda"))
    with pytest.raises(B.PrnError):   # offsets on the host are looked at
        prn.gated_scan(x[:1], cell="glr", cu_seqlens=[0, 3])
    with pytest.raises(ValueError):
        prn.gated_scan_backward(H[:, :3], x, H, cell="glr")
    with pytest.raises(ValueError):
        prn.gated_scan_backward(H, x, H, cell="glr", dstate=torch.zeros(1, 1, 8, device="cuda"))
    with pytest.raises(B.PrnUnsupportedError):
        prn.sequential_forward(x, torch.zeros(2, 8, device="cuda"), cell="glr")
    with pytest.raises(B.PrnError, match="gated linear cells"):
        prn.newton_forward(x, torch.zeros(2, 8, device="cuda"), 2, cell="glr")


@pytest.mark.parametrize("cu", [None, [0, 5, 4000001, 4300007]])
def test_offsets_past_32_bits(cu):
    """4300007 steps of 2 x 258 values: past the start, the last steps are those of a call that begins there."""
    T, d, cut = 4300007, 258, 4200000
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, T, 2, d, generator=g, device="cuda", dtype=torch.bfloat16)
    dH = torch.randn(1, T, d, generator=g, device="cuda", dtype=torch.bfloat16)
    x[:, cut - 1, 0] = -200.0   # this step's state is its input: what came before has no part in what follows
    if cu is not None:
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    H, last = prn.gated_scan(x, cell="glr", cu_seqlens=cu, return_state=True)
    dx, _ = prn.gated_scan_backward(dH, x, H, cell="glr", cu_seqlens=cu)
    end = slice(cut - 1, T)
    y, e = x[:, end].contiguous(), dH[:, end].contiguous()
    want, want_last = prn.gated_scan(y, cell="glr", return_state=True)
    want_dx, _ = prn.gated_scan_backward(e, y, want, cell="glr")
    # the chunks begin elsewhere: fp32 maps in another order, a bf16 value next to the other's
    near = lambda got, ref: (got.double() - ref.double()).abs() - 2.0 ** -7 * ref.double().abs()   # noqa: E731
    got_dx, want_dx = dx[:, end][:, 1:], want_dx[:, 1:]
    for got, ref in ((H[:, end], want), (last[-1:], want_last), (got_dx[:, :, 1], want_dx[:, :, 1])):
        assert (near(got, ref) <= 2.0 ** -12).all()
    # dx_f = lam (h - v) f (1 - f), h off by half a step of the state that its chunk starts from, in either call
    off = torch.sigmoid(-y[:, 1:, 0].double())
    lam = want_dx[:, :, 1].double().abs() / off
    bound = 2 * HALF[torch.bfloat16] * want.double().abs().max() * lam * off * (1 - off) * 1.01 + 2.0 ** -12
    assert (near(got_dx[:, :, 0], want_dx[:, :, 0]) <= bound).all()


# ------------------------------------------------------------------ gates at their ends ---

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cell", ["glr", "glri"])
@pytest.mark.parametrize("h0", [False, True])
@pytest.mark.parametrize("cu,T", [(None, 1), (None, 40), (None, 3000), ([0, 7, 7, 40], 40), ([0, 1, 1000, 3000], 3000)])
def test_a_gate_that_is_nan(cu, T, h0, cell, dtype):
    """A NaN forget gate at a sequence's first step or inside one: NaN where the definition has it, in states, final
    states and gradients, whatever the layout, and every other value to the bit."""
    for at in sorted({0, T // 2, T - 1, *(cu[:-1] if cu else ())}):
        c = _case(cell, 1, T, 40, dtype, cu, h0=h0, seed=at)
        kw = dict(cell=cell, h0=c["h0"], cu_seqlens=c["cu"])
        H, last = prn.gated_scan(c["x"], return_state=True, **kw)
        dx, dh0 = prn.gated_scan_backward(c["dH"], c["x"], H, dstate=c["dlast"], **kw)
        x = c["x"].clone()
        x[0, at, 0, 11] = float("nan")
        H2, last2 = prn.gated_scan(x, return_state=True, **kw)
        dx2, dh2 = prn.gated_scan_backward(c["dH"], x, H2, dstate=c["dlast"], **kw)
        want_H, want_last = gated.gated_scan(cell, _np(x), _np(c["h0"]), cu)
        want_dx, want_dh0 = gated.gated_scan_backward(cell, _np(x), _np(c["dH"]), _np(c["h0"]), cu, _np(c["dlast"]))
        assert np.isnan(want_H[0, at, 11])
        for name, got, clean, want in (("H", H2, H, want_H), ("last", last2, last, want_last), ("dxproj", dx2, dx, want_dx),
                                       ("dh0", dh2, dh0, want_dh0)):
            if got is None:
                continue
            nan = torch.from_numpy(np.isnan(want)).cuda()
            assert torch.equal(torch.isnan(got), nan), (name, at)
            assert torch.equal(got[~nan], clean[~nan]), (name, at)


def _nearly_shut(dtype):
    """Logits of gates from 1.6e-38 (a normal number) down to 0, through those whose value is no normal fp32 number,
    and which are those: from log(2^-126) = -87.3365 on."""
    x = torch.tensor([-87.0, -87.25, -87.375, -87.5, -87.75, -88.0, -88.25, -88.5, -88.6875, -88.71875, -88.75, -89.0, -100.0, -104.0])
    x = x.to(dtype).cuda()
    return x, x < -87.3366


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1, 20, 3000])
def test_gates_too_small_for_a_normal_number(T, dtype):
    """Where s(x_f) is below fp32's normal numbers 1 - s(x_f) is 1: the state is the input and the input's gradient
    the state's, exactly (what is kept of a state of order one is below 2^-125, far below half a step).  The logits
    before have 1 - s from a power and a quotient, within the oracle's bounds."""
    xf, shut = _nearly_shut(dtype)
    g = torch.Generator().manual_seed(T)
    v = torch.randn(1, T, len(xf), generator=g).to(dtype).cuda()
    x = torch.stack([xf.expand_as(v), v], 2).contiguous()
    h0 = torch.ones(1, 1, len(xf), dtype=dtype, device="cuda")
    dH = torch.randn(1, T, len(xf), generator=g).to(dtype).cuda()
    pack = torch.tensor([0, T // 2, T], dtype=torch.int32, device="cuda")
    H = prn.gated_scan(x, cell="glr", h0=h0)
    for got in (H, prn.gated_scan(x, cell="glr", cu_seqlens=pack)):
        assert torch.equal(got[..., shut], v[..., shut]), xf[(got != v).any(1)[0]]
    dx, dh0 = prn.gated_scan_backward(dH, x, H, cell="glr", h0=h0)
    assert torch.equal(dx[:, :, 1][..., shut], dH[..., shut])
    want_dx, want_dh0 = gated.gated_scan_backward("glr", _np(x), _np(dH), _np(h0))
    bounds = gated.gated_scan_bounds("glr", _np(x), _np(h0), None, _np(dH), start=HALF[dtype] / U24)
    for name, got, want in (("H", H, gated.gated_scan("glr", _np(x), _np(h0))[0]), ("dxproj", dx, want_dx), ("dh0", dh0, want_dh0)):
        _close(name, got, want, bounds[name], dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_step_whose_gate_is_too_small_for_a_normal_number(dtype):
    xf, shut = _nearly_shut(dtype)
    v = torch.linspace(-2.0, 2.0, len(xf)).to(dtype).cuda()
    W = torch.cat([xf, v])[:, None].contiguous()
    x = torch.ones(3, 1, dtype=dtype, device="cuda")
    out = torch.empty(3, 1, len(xf), dtype=dtype, device="cuda")
    B.prn_decode_step(x, W, None, None, out, cell="glr", state_in=torch.ones_like(out))
    want = v.expand_as(out)
    assert torch.equal(out[..., shut], want[..., shut])
    z, one = torch.stack([xf, v]).expand(3, 1, 2, len(xf)), np.ones((3, 1, len(xf)))
    _close("state", out, gated.gated_scan("glr", _np(z), one)[1], gated.gated_scan_bounds("glr", _np(z), one)["last"], dtype)


# ------------------------------------------------------------------ projections in bf16 ---

@pytest.mark.parametrize("cell", ["glr", "glri"])
@pytest.mark.parametrize("Bn,T,d_in,d", [(2, 50, 32, 24), (1, 300, 72, 40), (3, 129, 16, 7), (1, 4096, 64, 128)])
def test_projection_in_bf16_both_ways(cell, Bn, T, d_in, d):
    """Products of bf16 values are exact in fp32, a sum of n of them is off by (n + 8) 2^-24 of their magnitudes, and
    every result but the bias's gradient is rounded once to bf16."""
    g = torch.Generator().manual_seed(T)
    new = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    x, W = new(Bn, T, d_in).bfloat16().cuda().requires_grad_(), (new(G[cell] * d, d_in) / d_in ** 0.5).bfloat16().cuda().requires_grad_()
    bias, dz = new(G[cell] * d).cuda().requires_grad_(), new(Bn, T, G[cell], d).bfloat16().cuda()
    z = prn.input_proj_apply(x, W, bias, cell=cell)
    dx, dW, db = torch.autograd.grad(z, (x, W, bias), dz)
    M = Bn * T
    xd, Wd, bd, dzd = _np(x).reshape(M, -1), _np(W), _np(bias), _np(dz).reshape(M, -1)
    ax, aW, adz = np.abs(xd), np.abs(Wd), np.abs(dzd)
    for name, got, want, size, n, dtype in (
            ("z", z, xd @ Wd.T + bd, ax @ aW.T + np.abs(bd), d_in + 1, torch.bfloat16),
            ("dx", dx, dzd @ Wd, adz @ aW, G[cell] * d, torch.bfloat16),
            ("dW", dW, dzd.T @ xd, adz.T @ ax, M, torch.bfloat16),
            ("dbias", db, dzd.sum(0), adz.sum(0), M, torch.float32)):
        _close(name, got.reshape(want.shape), want, (n + 8) * size, dtype)
