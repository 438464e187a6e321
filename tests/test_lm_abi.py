"""CPU-only checks of the token-model entry points: struct layouts, workspace
sizes, and refusals before anything is launched."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from nonlinear_rnn_amd import binding as B
from nonlinear_rnn_amd import lm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libprn.so not built")

FAKE = 1 << 20   # an aligned non-null address; never dereferenced
BAD, UNSUP, WS = B.PRN_ERR_INVALID_ARG, B.PRN_ERR_UNSUPPORTED, B.PRN_ERR_WORKSPACE
STRUCTS = ("prn_embed_params", "prn_block_norm_params", "prn_vocab_loss_params")


def test_struct_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines, want = [], []
    for s in STRUCTS:
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
    p = cls(**{**base, **kw})
    return ctypes.byref(p)


EMBED = dict(dtype=0, token_bytes=8, N=10, V=20, d=16, scale=1.0, pad_id=B.NO_PAD)
NORM = dict(dtype=0, act=0, N=10, d=16, eps=1e-6)
LOSS = dict(dtype=0, target_bytes=8, N=10, V=20, d=16, scale=1.0, ignore_index=-100)


@pytest.mark.parametrize("kw,args,status", [
    (dict(dtype=2), {}, BAD), (dict(token_bytes=2), {}, BAD), (dict(N=-1), {}, BAD), (dict(V=0), {}, BAD),
    (dict(d=0), {}, BAD), (dict(N=1 << 31), {}, UNSUP), (dict(V=(1 << 31) - 1), {}, UNSUP),
    (dict(), dict(tokens=None), BAD), (dict(), dict(rows=None), BAD), (dict(), dict(out=None), BAD),
    (dict(), dict(tokens=FAKE + 4), BAD), (dict(), dict(rows=FAKE + 2), BAD),
])
def test_embed_refusals(kw, args, status):
    a = dict(tokens=FAKE, rows=FAKE, out=FAKE)
    a.update(args)
    L = B.lib()
    assert L.prn_embed(a["tokens"], a["rows"], _p(B.prn_embed_params, EMBED, **kw), a["out"]) == status
    assert B.prn_last_error()
    assert L.prn_embed_backward(a["tokens"], a["rows"], _p(B.prn_embed_params, EMBED, **kw), a["out"]) == status
    assert B.prn_last_error()


def test_embed_backward_needs_its_workspace_and_an_aligned_table():
    L = B.lib()
    assert L.prn_embed_backward(FAKE, FAKE, _p(B.prn_embed_params, EMBED), FAKE) == WS
    assert L.prn_embed_backward(FAKE, FAKE, _p(B.prn_embed_params, EMBED), FAKE + 8) == BAD
    n = B.prn_embed_backward_workspace_bytes(torch.float32, 10, 20, 16)
    kw = dict(workspace=FAKE + 4, workspace_bytes=n)
    assert L.prn_embed_backward(FAKE, FAKE, _p(B.prn_embed_params, EMBED, **kw), FAKE) == WS
    assert B.prn_embed_backward_workspace_bytes(torch.float32, 0, 20, 16) == 0
    assert L.prn_embed_backward(FAKE, FAKE, None, FAKE) == BAD
    with pytest.raises(B.PrnError):
        B.prn_embed_backward_workspace_bytes(torch.float32, -1, 20, 16)


@pytest.mark.parametrize("kw,args,status", [
    (dict(dtype=2), {}, BAD), (dict(act=2), {}, BAD), (dict(N=-1), {}, BAD), (dict(d=0), {}, BAD),
    (dict(d=8193), {}, UNSUP), (dict(N=1 << 31), {}, UNSUP), (dict(eps=-1.0), {}, BAD), (dict(eps=float("nan")), {}, BAD),
    (dict(w_post=FAKE + 2), {}, BAD), (dict(), dict(h=None), BAD), (dict(), dict(h=FAKE + 8), BAD),
    (dict(), dict(gate=FAKE + 4), BAD), (dict(), dict(x=FAKE + 4), BAD),
    (dict(w_pre=FAKE), {}, BAD),                 # no n_out / dn
    (dict(), dict(n=FAKE), BAD),                 # n_out / dn without w_pre
])
def test_block_norm_refusals(kw, args, status):
    a = dict(h=FAKE, gate=None, x=None, r=FAKE, n=None)
    a.update(args)
    L = B.lib()
    assert L.prn_block_norm(a["h"], a["gate"], a["x"], _p(B.prn_block_norm_params, NORM, **kw), a["r"],
                            a["n"]) == status
    assert B.prn_last_error()
    st = L.prn_block_norm_backward(a["h"], a["gate"], a["x"], a["r"], a["n"], _p(B.prn_block_norm_params, NORM, **kw),
                                   FAKE, None, None, None, None, None)
    assert st == status, B.prn_last_error()


def test_block_norm_refuses_missing_outputs_and_gradients_of_absent_inputs():
    L, P = B.lib(), B.prn_block_norm_params
    assert L.prn_block_norm(FAKE, None, None, _p(P, NORM), None, None) == BAD
    ws = dict(workspace=FAKE, workspace_bytes=1 << 40)
    for k in range(1, 6):
        outs = [FAKE, None, None, None, None, None]
        outs[k] = FAKE
        assert L.prn_block_norm_backward(FAKE, None, None, FAKE, None, _p(P, NORM, **ws), *outs) == BAD
        assert "absent" in B.prn_last_error()
    assert L.prn_block_norm_backward(FAKE, None, None, FAKE, None, _p(P, NORM), FAKE, *[None] * 5) == WS


@pytest.mark.parametrize("kw,args,status", [
    (dict(dtype=2), {}, BAD), (dict(target_bytes=1), {}, BAD), (dict(N=-1), {}, BAD), (dict(V=0), {}, BAD),
    (dict(d=0), {}, BAD), (dict(N=1 << 31), {}, UNSUP), (dict(V=1 << 31), {}, UNSUP), (dict(d=1 << 20), {}, UNSUP),
    (dict(scale=0.0), {}, BAD), (dict(scale=-1.0), {}, BAD), (dict(scale=float("inf")), {}, BAD),
    (dict(N=(1 << 31) - 1, V=1 << 30), {}, UNSUP),
    (dict(), dict(x=None), BAD), (dict(), dict(W=None), BAD), (dict(), dict(t=None), BAD), (dict(), dict(a=None), BAD),
    (dict(), dict(b=None), BAD), (dict(), dict(x=FAKE + 8), BAD), (dict(), dict(W=FAKE + 8), BAD),
    (dict(), dict(t=FAKE + 4), BAD), (dict(), dict(a=FAKE + 2), BAD),
    (dict(), {}, WS), (dict(workspace=FAKE, workspace_bytes=16), {}, WS),
    (dict(workspace=FAKE + 16, workspace_bytes=1 << 40), {}, WS),
])
def test_vocab_loss_refusals(kw, args, status):
    a = dict(x=FAKE, W=FAKE, t=FAKE, a=FAKE, b=FAKE)
    a.update(args)
    L, P = B.lib(), B.prn_vocab_loss_params
    assert L.prn_vocab_loss(a["x"], a["W"], a["t"], _p(P, LOSS, **kw), a["a"], a["b"]) == status, B.prn_last_error()
    assert B.prn_last_error()
    st = L.prn_vocab_loss_backward(a["x"], a["W"], a["t"], a["a"], a["b"], None, _p(P, LOSS, **kw), FAKE, FAKE)
    assert st == status, B.prn_last_error()


def test_workspace_sizes_are_sane():
    """The loss's workspace does not grow with N x V."""
    small = B.prn_vocab_loss_workspace_bytes(torch.bfloat16, 32768, 32768, 512)
    assert 0 < small < 64 << 20
    back = B.prn_vocab_loss_backward_workspace_bytes(torch.bfloat16, 32768, 131072, 512)
    assert 0 < back < 1200 << 20
    assert B.prn_vocab_loss_workspace_bytes(torch.float32, 0, 100, 8) == 0
    with pytest.raises(B.PrnError):
        B.prn_vocab_loss_workspace_bytes(torch.float32, 4, 0, 8)
    with pytest.raises(TypeError):
        B.prn_vocab_loss_workspace_bytes(torch.float16, 4, 4, 8)


def test_python_refusals_without_a_gpu():
    """Tensors that are not on a GPU, wrong types and shapes are refused before the library is called."""
    cpu = torch.zeros(4, 8)
    ids = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError):
        lm.embed(ids, cpu)
    with pytest.raises(TypeError):
        lm.block_norm(cpu, w_pre=torch.ones(8))
    with pytest.raises(ValueError):
        lm.block_norm(cpu)
    with pytest.raises(TypeError):
        lm.vocab_loss(cpu, cpu, ids)
    with pytest.raises(ValueError):
        lm.embed_backward(torch.zeros(3, 8), ids, 4)


def test_tensors_of_as_many_rows_in_another_order_are_refused():
    """Rows are flattened: a (T, B) tensor beside a (B, T) one would pair the wrong rows."""
    x, W, t = torch.zeros(2, 3, 8), torch.zeros(5, 8), torch.zeros(3, 2, dtype=torch.int64)
    good = torch.zeros(2, 3, dtype=torch.int64)
    for call in (lambda: lm.vocab_loss(x, W, t), lambda: lm.vocab_loss(x, W, good.view(-1)),
                 lambda: lm.vocab_loss(x, W.view(5, 1, 8), good), lambda: lm.vocab_loss_apply(x, W, t)):
        with pytest.raises(ValueError):
            call()
    f = torch.zeros(2, 3)
    for dloss, targets, lse, dlse in ((f.t(), good, f, None), (f, t, f, None), (f, good, f.t(), None), (f, good, f, f.t())):
        with pytest.raises(ValueError):
            lm.vocab_loss_backward(dloss, x, W, targets, lse, dlse=dlse)
    y, w = x.transpose(0, 1), torch.ones(8)
    for call in (lambda: lm.block_norm(x, y), lambda: lm.block_norm(x, gate=y), lambda: lm.block_norm_apply(x, y, w_pre=w),
                 lambda: lm.block_norm_backward(y, None, x, gate=x), lambda: lm.block_norm_backward(None, y, x, w_pre=w),
                 lambda: lm.block_norm_backward(x, None, x, y), lambda: lm.block_norm_backward(x, None, x, gate=y)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        lm.embed_backward(y, good, 5)
