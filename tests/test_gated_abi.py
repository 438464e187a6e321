"""CPU-only checks of the linear-recurrence block's entry points: struct
layouts, workspace sizes, and refusals before anything is launched."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import nonlinear_rnn_amd as prn
from nonlinear_rnn_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libprn.so not built")

FAKE = 1 << 20   # an aligned non-null address; never dereferenced
BAD, UNSUP, WS = B.PRN_ERR_INVALID_ARG, B.PRN_ERR_UNSUPPORTED, B.PRN_ERR_WORKSPACE
BIG = dict(workspace=FAKE, workspace_bytes=1 << 60)


def test_struct_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines, want = [], []
    for s in ("prn_gated_ffn_params", "prn_dropout_params"):
        cls = getattr(B, s)
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({s}, {f}));')
            want.append(getattr(cls, f).offset)
        lines.append(f'printf("%zu\\n", sizeof({s}));')
        want.append(ctypes.sizeof(cls))
    src = tmp_path / "off.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "prn.h"\nint main(void){\n' + "\n".join(lines)
                   + "return 0;}\n")
    exe = tmp_path / "off"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == want


def _p(cls, base, **kw):
    return ctypes.byref(cls(**{**base, **kw}))


SCAN = dict(cell=2, dtype=0, B=2, T=1000, d_h=16, n_seqs=0)
FFN = dict(dtype=0, act=0, N=10, d=16, F=8)
DROP = dict(dtype=0, n=100, p=0.5, seed=1, offset=2)


@pytest.mark.parametrize("kw,args,status", [
    (dict(cell=0), {}, UNSUP), (dict(cell=1), {}, UNSUP), (dict(cell=9), {}, BAD), (dict(dtype=2), {}, BAD),
    (dict(B=0), {}, BAD), (dict(T=-1), {}, BAD), (dict(d_h=0), {}, BAD), (dict(n_seqs=-1), {}, BAD),
    (dict(T=1 << 31), {}, UNSUP), (dict(n_seqs=3), dict(cu=FAKE), BAD), (dict(n_seqs=3, B=1), {}, BAD),
    (dict(), dict(cu=FAKE), BAD), (dict(n_seqs=3, B=1), dict(cu=FAKE + 2), BAD), (dict(), dict(x=None), BAD),
    (dict(), dict(H=None), BAD), (dict(), dict(x=FAKE + 8), BAD), (dict(), dict(h0=FAKE + 4), BAD),
    (dict(), dict(H=FAKE + 4), BAD), (dict(workspace=None, workspace_bytes=0), {}, WS),
    (dict(workspace_bytes=8), {}, WS), (dict(workspace=FAKE + 16), {}, WS),
])
def test_scan_refusals(kw, args, status):
    a = dict(x=FAKE, h0=None, cu=None, H=FAKE)
    a.update(args)
    L, base = B.lib(), {**SCAN, **BIG}
    assert L.prn_gated_scan(a["x"], _p(B.prn_params, base, **kw), a["h0"], a["cu"], a["H"]) == status, B.prn_last_error()
    assert B.prn_last_error()
    st = L.prn_gated_scan_backward(a["x"], _p(B.prn_params, base, **kw), a["h0"], a["cu"], a["H"], FAKE, None, FAKE, None)
    assert st == status, B.prn_last_error()


def test_scan_backward_refuses_missing_and_unaligned_tensors():
    L = B.lib()
    for k in range(4):
        for v in (None, FAKE + 8):
            if k == 1 and v is None:
                continue   # no gradient of the final states
            t = [FAKE, None, FAKE, None]   # dH, dstate_last, dxproj, dh0
            t[k] = v
            if k == 3 and v is None:
                continue
            assert L.prn_gated_scan_backward(FAKE, _p(B.prn_params, {**SCAN, **BIG}), None, None, FAKE, *t) == BAD
    assert L.prn_gated_scan(FAKE, None, None, None, FAKE) == BAD


def test_the_newton_entry_points_refuse_the_gated_cells():
    L = B.lib()
    p = lambda **kw: _p(B.prn_params, {**SCAN, **BIG, "a": FAKE}, **kw)   # noqa: E731
    for cell in (2, 3):
        assert L.prn_newton_forward(FAKE, p(cell=cell), None, 2, None, FAKE, None) == UNSUP
        assert L.prn_sequential_forward(FAKE, p(cell=cell), None, None, FAKE) == UNSUP
        assert L.prn_newton_backward(FAKE, p(cell=cell), None, None, FAKE, FAKE, None, FAKE, FAKE, None) == UNSUP
        assert L.prn_newton_forward_noalloc(FAKE, p(cell=cell), None, 2, None, FAKE, None) == UNSUP
        assert L.prn_head_sequential_forward(FAKE, p(cell=cell), FAKE, 16, None, FAKE) == UNSUP
        assert L.prn_workspace_bytes(p(cell=cell), 2) == 0 and "gated" in B.prn_last_error()
        # a decode step of them needs no recurrent weights, one of the others does
        assert L.prn_decode_step(FAKE, None, None, p(cell=cell, T=1, d_in=8, a=None), None, FAKE, None) == BAD
        assert L.prn_decode_step(FAKE, FAKE, None, p(cell=cell, T=2, d_in=8, a=None), None, FAKE, None) == BAD
    assert L.prn_decode_step(FAKE, FAKE, None, p(cell=0, T=1, d_in=8, a=None), None, FAKE, None) == BAD


@pytest.mark.parametrize("kw,args,status", [
    (dict(dtype=2), {}, BAD), (dict(act=2), {}, BAD), (dict(N=-1), {}, BAD), (dict(d=0), {}, BAD), (dict(F=0), {}, BAD),
    (dict(N=1 << 31), {}, UNSUP), (dict(F=1 << 20, d=1 << 12), {}, UNSUP), (dict(N=(1 << 31) - 1, F=1 << 10), {}, UNSUP),
    (dict(), dict(x=None), BAD), (dict(), dict(W=None), BAD), (dict(), dict(g=None), BAD), (dict(), dict(x=FAKE + 8), BAD),
    (dict(), dict(W=FAKE + 4), BAD), (dict(), dict(g=FAKE + 2), BAD),
    (dict(N=1000, F=800, d=7, workspace=None, workspace_bytes=0), {}, WS), (dict(N=1000, F=800, d=7, workspace_bytes=64), {}, WS),
    (dict(N=1000, F=800, d=7, workspace=FAKE + 16), {}, WS),
])
def test_ffn_refusals(kw, args, status):
    a = dict(x=FAKE, W=FAKE, g=FAKE)
    a.update(args)
    L, base = B.lib(), {**FFN, **BIG}
    assert L.prn_gated_ffn(a["x"], a["W"], _p(B.prn_gated_ffn_params, base, **kw), a["g"]) == status, B.prn_last_error()
    assert B.prn_last_error()
    st = L.prn_gated_ffn_backward(a["x"], a["W"], a["g"], _p(B.prn_gated_ffn_params, base, **kw), FAKE, FAKE)
    assert st == status, B.prn_last_error()


def test_ffn_backward_refuses_unaligned_gradients():
    L, p = B.lib(), _p(B.prn_gated_ffn_params, {**FFN, **BIG})
    assert L.prn_gated_ffn_backward(FAKE, FAKE, FAKE, p, FAKE + 8, None) == BAD
    assert L.prn_gated_ffn_backward(FAKE, FAKE, FAKE, p, None, FAKE + 8) == BAD
    assert L.prn_gated_ffn_backward(FAKE, FAKE, FAKE, _p(B.prn_gated_ffn_params, FFN), FAKE, None) == WS
    assert L.prn_gated_ffn(FAKE, FAKE, None, FAKE) == BAD


@pytest.mark.parametrize("kw,args", [
    (dict(dtype=2), {}), (dict(n=-1), {}), (dict(n=1 << 41), {}), (dict(p=-0.01), {}), (dict(p=1.01), {}),
    (dict(p=float("nan")), {}), (dict(), dict(x=None)), (dict(), dict(out=None)), (dict(), dict(x=FAKE + 8)),
    (dict(), dict(r=FAKE + 8)), (dict(), dict(out=FAKE + 4)), (dict(state=FAKE + 4), {}),
])
def test_dropout_refusals(kw, args):
    a = dict(x=FAKE, r=None, out=FAKE)
    a.update(args)
    assert B.lib().prn_dropout(a["x"], a["r"], _p(B.prn_dropout_params, DROP, **kw), a["out"]) == BAD
    assert B.prn_last_error()
    assert B.lib().prn_dropout(FAKE, None, None, FAKE) == BAD


def test_workspace_sizes():
    """A scan's workspace is the maps of its ranges, a few MB at most; none where a range is the whole row."""
    for cell in ("glr", "glri"):
        assert B.prn_gated_scan_workspace_bytes(cell, torch.float32, 4, 1, 100) == 0
        assert B.prn_gated_scan_workspace_bytes(cell, torch.float32, 4, 0, 100) == 0
        assert 0 < B.prn_gated_scan_workspace_bytes(cell, torch.float32, 2, 131072, 256) < 8 << 20
        assert 0 < B.prn_gated_scan_backward_workspace_bytes(cell, torch.bfloat16, 1, 100000, 64, 7) < 8 << 20
    for cell, rows in (("gru", 4), ("glr", 0)):
        with pytest.raises(B.PrnError):
            B.prn_gated_scan_workspace_bytes(cell, torch.float32, rows, 8, 8)
    assert B.prn_gated_ffn_workspace_bytes(torch.float32, 0, 7, 8) == 0
    assert B.prn_gated_ffn_backward_workspace_bytes(torch.bfloat16, 1000, 512, 2048) >= 1000 * 2 * 2048 * 2
    with pytest.raises(B.PrnError):
        B.prn_gated_ffn_workspace_bytes(torch.float32, 4, 0, 8)


def test_python_refusals_without_a_gpu():
    x = torch.zeros(2, 4, 2, 8)
    with pytest.raises(TypeError):
        prn.gated_scan(x, cell="glr")
    with pytest.raises(TypeError):
        prn.gated_ffn(torch.zeros(4, 8), torch.zeros(6, 8))
    with pytest.raises(ValueError):
        prn.gated_ffn(torch.zeros(4, 8), torch.zeros(5, 8))
    with pytest.raises(ValueError):
        prn.gated_ffn_backward(torch.zeros(3, 4), torch.zeros(4, 8), torch.zeros(6, 8))
    with pytest.raises(TypeError):
        prn.dropout(torch.zeros(8), 0.5, seed=1)
    with pytest.raises(ValueError):
        prn.dropout(torch.zeros(8), 0.5, seed=1, residual=torch.zeros(2, 4))


def test_no_table_of_iterations_for_the_gated_cells():
    from nonlinear_rnn_amd import kstar
    with pytest.raises(ValueError, match="no table"):
        kstar.load_table("glr")


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("N,d,F", [(256, 64, 5000000), (256, 128, 4300000), (128, 32, 9000000), (4096, 1, 1 << 22),
                                   (256, 64, (1 << 22) - 63)])
def test_ffn_gradients_of_rows_past_32_bits(N, d, F, dtype):
    """A tile of dx reads up to 256 rows of dz, of 4 (F + 64) bytes each at most, by offsets of 32 bits: past them
    the gradients are refused, the product itself is not."""
    L, p = B.lib(), _p(B.prn_gated_ffn_params, {**FFN, **BIG}, N=N, d=d, F=F, dtype=dtype)
    assert L.prn_gated_ffn_backward(FAKE, FAKE, FAKE, p, FAKE, FAKE) == UNSUP and "2^30" in B.prn_last_error()
    with pytest.raises(B.PrnError, match="2\\^30"):
        B.prn_gated_ffn_backward_workspace_bytes((torch.float32, torch.bfloat16)[dtype], N, d, F)
    L.prn_gated_ffn_workspace_bytes(p)
    assert B.prn_last_error() == ""


@pytest.mark.parametrize("N,d,F", [(256, 64, (1 << 22) - 64), (100, 32, 9000000), (1, 32, 9000000)])
def test_ffn_gradients_of_rows_within_32_bits(N, d, F):
    assert min(N, 256) * 2 * (2 * ((F + 31) // 32 * 32) + 64) < 1 << 32   # rows of both halves, in blocks of 32, and 64 between
    for dtype in (torch.float32, torch.bfloat16):
        assert B.prn_gated_ffn_backward_workspace_bytes(dtype, N, d, F) > N * 4 * F


@pytest.mark.parametrize("N,d,F", [(1 << 30, 32, 32), ((1 << 31) - 1, 1, 1), (1 << 26, 32, 1 << 11), (1 << 26, 1 << 11, 32),
                                   ((1 << 37) // 256 - 256, 128, 16), ((1 << 37) // 129 - 255, 1, 1)])
def test_ffn_refuses_the_rows_that_its_limits_name(N, d, F):
    """Both ways refuse (N + 256) (F + 128) or (N + 256) (d + 128) of 2^37 on, and say so; the size before is taken."""
    L = B.lib()
    widest = max(d, F) + 128
    assert (N + 256) * widest >= 1 << 37
    p = _p(B.prn_gated_ffn_params, {**FFN, **BIG}, N=N, d=d, F=F)
    assert L.prn_gated_ffn(FAKE, FAKE, p, FAKE) == UNSUP and "2^37" in B.prn_last_error()
    assert L.prn_gated_ffn_backward(FAKE, FAKE, FAKE, p, FAKE, FAKE) == UNSUP and "2^37" in B.prn_last_error()
    most = ((1 << 37) - 1) // widest - 256
    for dtype in (torch.float32, torch.bfloat16):
        B.prn_gated_ffn_workspace_bytes(dtype, most, d, F)
        assert B.prn_gated_ffn_backward_workspace_bytes(dtype, most, d, F) > most * 4 * F
