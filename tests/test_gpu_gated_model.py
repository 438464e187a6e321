"""The linear-recurrence model of examples/token_model.py, the operators as they
are used together: its gradients against the same model in float64 PyTorch on
the CPU (with the same dropout), its serving step against its training forward,
a ragged pack against its sequences, and a captured training step.

Tolerances.  fp32, two layers, d = 48: as in the recurrent model's test, every
operator holds its own result to a few 1e-6 relative and the longest path
passes about twenty of them each way: 40 x 5e-6, doubled for the softmax's
sensitivity to its logits (of order one): 4e-4, relative to the parameter's
largest gradient entry.  Scores are compared absolutely, log probabilities of
order ten: 4e-4 as well.
"""
import importlib.util
import os

import pytest
import torch

from oracle import gated

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "token_model.py")
TOL = 4e-4


def _example():
    spec = importlib.util.spec_from_file_location("token_model", _PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _model(ex, cell, p, seed=1, V=97, width=48):
    torch.manual_seed(seed)
    return ex.LinearTokenModel(V, width, 2, 70, p, cell)


def _plain(model, tokens, seed, step):
    """The same features in float64; parameters by the model's names."""
    q = {k: v.detach().double().cpu().requires_grad_() for k, v in model.named_parameters()}
    d, pad, lin = model.width, model.pad, torch.nn.functional.linear
    rms = lambda y: y * (y.square().mean(-1, keepdim=True) + 1e-6).rsqrt()   # noqa: E731
    x = q["table"][tokens] * d ** 0.5 * (tokens != pad).unsqueeze(-1)
    for i in range(len(model.layers)):
        w = {k.split(".", 2)[2]: v for k, v in q.items() if k.startswith(f"layers.{i}.")}
        n = rms(x) * w["w_pre"]
        z = (n @ w["W"].T + w["bias"]).view(*n.shape[:2], -1, d)
        f, v = torch.sigmoid(z[:, :, 0]), z[:, :, -1]
        u = (1 - f) * v if model.cell == "glr" else torch.sigmoid(z[:, :, 1]) * v
        h, hs = torch.zeros(n.shape[0], d, dtype=torch.float64), []
        for t in range(n.shape[1]):
            h = f[:, t] * h + u[:, t]
            hs.append(h)
        x = x + w["alpha"] * rms(torch.stack(hs, 1)) * w["w_post"] * torch.nn.functional.silu(lin(n, w["Wg"]))
        g, up = lin(rms(x) * w["w_ffn"], w["Wf"]).chunk(2, -1)
        y = lin(torch.nn.functional.silu(g) * up, w["Wd"])
        if seed is not None:
            keep = torch.from_numpy(gated.kept(y.numel(), model.p, seed, step * len(model.layers) + i)).view(y.shape)
            y = y * keep / (1 - round(model.p * 65536) / 65536)
        x = x + y
    return rms(x) * q["w_out"], q


@pytest.mark.parametrize("cell", ["glr", "glri"])
def test_gradients_match_float64(cell):
    ex = _example()
    model = _model(ex, cell, 0.25)
    tokens, targets = ex.chain(3, 40, 97, torch.Generator(device="cuda").manual_seed(2))
    tokens[1, 30:] = model.pad
    targets[1, 29:] = model.pad
    loss = model.loss(tokens, targets, seed=5, step=3)
    loss.backward()
    n, q = _plain(model, tokens.cpu(), 5, 3)
    t = targets.cpu()
    logits = n @ q["table"].T
    each = (torch.logsumexp(logits, -1) - logits.gather(-1, t.unsqueeze(-1))[..., 0]) * (t != model.pad)
    want = each.sum() / (t != model.pad).sum()
    want.backward()
    assert abs(loss.item() - want.item()) <= TOL
    for name, p in model.named_parameters():
        got, ref = p.grad.double().cpu(), q[name].grad
        err = ((got - ref).abs().max() / ref.abs().max()).item()
        print(f"  {name}: {err:.2e}", flush=True)
        assert err <= TOL, name


@pytest.mark.parametrize("cell", ["glr", "glri"])
def test_serving_matches_training_forward(cell):
    ex = _example()
    model = _model(ex, cell, 0.5, V=300, width=64)
    tokens, targets = ex.chain(5, 24, 300, torch.Generator(device="cuda").manual_seed(4))
    with torch.no_grad():
        loss, _ = ex.prn.vocab_loss(model.features(tokens), model.table, targets, ignore_index=model.pad)
    carry, scores = None, []
    for t in range(tokens.shape[1]):
        score, carry = model.step(tokens[:, t].contiguous(), carry, targets[:, t].contiguous())
        scores.append(score)
    assert (torch.stack(scores, 1) + loss).abs().max().item() <= TOL


def test_a_pack_matches_its_sequences():
    ex = _example()
    model = _model(ex, "glr", 0.0)
    tokens, _ = ex.chain(1, 400, 97, torch.Generator(device="cuda").manual_seed(3))
    cu = [0, 17, 17, 150, 151, 400]
    with torch.no_grad():
        whole = model.features(tokens, cu_seqlens=cu)
        for lo, hi in zip(cu[:-1], cu[1:]):
            if hi > lo:   # features of order one
                assert (whole[:, lo:hi] - model.features(tokens[:, lo:hi].contiguous())).abs().max().item() <= TOL


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_runs(dtype):
    ex = _example()
    torch.manual_seed(5)
    model = ex.LinearTokenModel(200, 64, 2, 96, 0.1, dtype=dtype)
    tokens, targets = ex.chain(8, 300, 200, torch.Generator(device="cuda").manual_seed(6))
    losses = [model.loss(tokens, targets, seed=s).item() for s in (9, 9, 10)]
    assert losses[0] == losses[1] != losses[2]   # the seed decides
    ex.train(model, tokens, targets, 3, seed=9)
    assert all(torch.isfinite(p.grad).all() for p in model.parameters())


def test_a_captured_training_step():
    """Forward, backward and an update in a graph, replayed on new tokens with new dropout numbers, against the same
    steps without one.  The eager steps run on a copy: no graph of these leaves lives beside the captured one."""
    ex = _example()
    prn = ex.prn
    gen = torch.Generator(device="cuda").manual_seed(8)

    def parts():
        torch.manual_seed(2)
        new = lambda *s: (torch.randn(*s, device="cuda") / 8).requires_grad_()   # noqa: E731
        return dict(W=new(2 * 64, 48), Wf=new(2 * 40, 64))

    def step(w, x, state):
        h = prn.gated_scan_apply(prn.input_proj_apply(x, w["W"], cell="glr"), cell="glr")
        y = prn.dropout_apply(prn.gated_ffn_apply(h, w["Wf"]), 0.25, seed=state)
        grads = torch.autograd.grad(y.square().mean(), list(w.values()))
        with torch.no_grad():
            for p, g in zip(w.values(), grads):
                p.sub_(g)
        return y

    held, eager = parts(), parts()
    x, state = torch.randn(2, 400, 48, device="cuda"), torch.tensor([4, 0], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(parts(), x, state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(held, x, state)
    for k in range(4):
        x.copy_(torch.randn(2, 400, 48, device="cuda", generator=gen))
        state[1] = k
        want = step(eager, x, state)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), k
        assert all(torch.equal(held[n], eager[n]) for n in held), k


def test_a_wait_that_gives_up_raises(monkeypatch):
    """PRN_SPIN_LIMIT=0: every wait of both passes gives up at once.  The call's error word is set, check_waits raises,
    and a training step ends there, with the weights as they were."""
    ex = _example()
    prn = ex.prn
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(1, 3000, 2, 64, generator=g, device="cuda").requires_grad_()
    words = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(3)]
    torch.manual_seed(7)
    model = ex.LinearTokenModel(100, 32, 1, 48)
    before = [p.detach().clone() for p in model.parameters()]
    tokens, targets = ex.chain(1, 1000, 100, g)
    H = prn.gated_scan_apply(x, cell="glr", error_out=words[0])
    torch.autograd.grad(H.sum(), x)
    prn.check_waits(words[0])

    H = prn.gated_scan_apply(x, cell="glr", error_out=words[0])
    monkeypatch.setenv("PRN_SPIN_LIMIT", "0")
    torch.autograd.grad(H.sum(), x)   # of the backward pass
    prn.gated_scan_apply(x, cell="glr", error_out=words[1])
    prn.gated_scan_backward(torch.ones_like(H), x.detach(), H.detach(), cell="glr", error_out=words[2])
    for word in words:
        with pytest.raises(prn.LookbackTimeoutError, match="gated_scan"):
            prn.check_waits(word)
    with pytest.raises(prn.LookbackTimeoutError):
        ex.train(model, tokens, targets, 2, seed=1)
    assert all(torch.equal(p, q) for p, q in zip(model.parameters(), before))
    monkeypatch.delenv("PRN_SPIN_LIMIT")
    model.waits.zero_()
    ex.train(model, tokens, targets, 2, seed=1)
