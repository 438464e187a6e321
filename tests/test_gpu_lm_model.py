"""The token model of examples/token_model.py: its gradients against the same
model in float64 PyTorch on the CPU, its serving step against its training
forward, and a few steps of training.

Tolerances.  fp32, two layers, d = 48: every operator holds its own result to
a few 1e-6 relative (their own tests); the longest path to a parameter passes
about twelve of them forward and as many backward, and the recurrence adds its
agreement bound of 1e-4 on h of order one.  Gradients are compared relative to
the parameter's largest gradient entry: 24 x 5e-6 + 1e-4, doubled for the
softmax's sensitivity to its logits (of order one): 5e-4.  Scores are
compared absolutely, log probabilities of order ten: 5e-4 as well.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "token_model.py")
TOL = 5e-4


def _example():
    spec = importlib.util.spec_from_file_location("token_model", _PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _plain_loss(model, tokens, targets, z_loss):
    """The same model in float64, sequentially unrolled; parameters by the model's names."""
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in model.named_parameters()}
    d, pad = model.width, model.pad
    def rms(y):
        return y * (y.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    x = p["table"][tokens] * d ** 0.5 * (tokens != pad).unsqueeze(-1)
    h = gate = None
    for i in range(len(model.layers) + 1):
        if i:
            q = f"layers.{i - 1}."
            x = x + p[q + "alpha"] * rms(h) * p[q + "w_post"] * torch.nn.functional.silu(gate)
        n = rms(x) * (p[f"layers.{i}.w_pre"] if i < len(model.layers) else p["w_out"])
        if i < len(model.layers):
            q = f"layers.{i}."
            gate = n @ p[q + "Wg"].T
            xp = (n @ p[q + "W"].T + p[q + "bias"]).view(*n.shape[:2], 3, d)
            az, ar, ac = p[q + "a"]
            s, hs = torch.zeros(n.shape[0], d, dtype=torch.float64), []
            for t in range(n.shape[1]):
                z, r = torch.sigmoid(az * s + xp[:, t, 0]), torch.sigmoid(ar * s + xp[:, t, 1])
                s = (1 - z) * s + z * torch.tanh(ac * (r * s) + xp[:, t, 2])
                hs.append(s)
            h = torch.stack(hs, 1)
    logits = n @ p["table"].T
    lse = torch.logsumexp(logits, -1)
    loss = (lse - logits.gather(-1, targets.unsqueeze(-1))[..., 0]) * (targets != pad)
    total = loss.sum() / (targets != pad).sum() + z_loss * lse.square().mean()
    return total, p


def test_gradients_match_float64():
    ex = _example()
    torch.manual_seed(1)
    model = ex.TokenModel(97, 48, 2)
    tokens, targets = ex.chain(3, 40, 97, torch.Generator(device="cuda").manual_seed(2))
    tokens[1, 30:] = model.pad
    targets[1, 29:] = model.pad
    loss = model.loss(tokens, targets, K=6, z_loss=1e-2)
    loss.backward()
    want, p = _plain_loss(model, tokens.cpu(), targets.cpu(), 1e-2)
    want.backward()
    assert abs(loss.item() - want.item()) <= TOL
    for name, q in model.named_parameters():
        got, ref = q.grad.double().cpu(), p[name].grad
        err = ((got - ref).abs().max() / ref.abs().max()).item()
        print(f"  {name}: {err:.2e}", flush=True)
        assert err <= TOL, name


def test_serving_matches_training_forward():
    ex = _example()
    torch.manual_seed(3)
    model = ex.TokenModel(300, 64, 2)
    tokens, targets = ex.chain(5, 24, 300, torch.Generator(device="cuda").manual_seed(4))
    with torch.no_grad():
        loss, _ = ex.prn.vocab_loss(model.features(tokens, K=6), model.table, targets, ignore_index=model.pad)
    carry, scores = None, []
    for t in range(tokens.shape[1]):
        score, carry = model.step(tokens[:, t].contiguous(), carry, targets[:, t].contiguous())
        scores.append(score)
    assert (torch.stack(scores, 1) + loss).abs().max().item() <= TOL


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_few_steps_learn(dtype):
    ex = _example()
    torch.manual_seed(5)
    model = ex.TokenModel(200, 64, 2, dtype)
    tokens, targets = ex.chain(8, 128, 200, torch.Generator(device="cuda").manual_seed(6))
    losses = ex.train(model, tokens, targets, 40)
    assert losses[-1] < 0.7 * losses[0]


def _losses():
    """(name, leaves, loss) of each differentiable operator."""
    import nonlinear_rnn_amd as prn
    g = torch.Generator(device="cuda").manual_seed(7)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda", requires_grad=True)   # noqa: E731
    ids = torch.randint(0, 30, (12,), generator=g, device="cuda")
    table, x, h, gate, w = new(30, 16), new(12, 16), new(12, 16), new(12, 16), new(16)
    yield "embed", (table,), lambda: prn.embed_apply(ids, table).square().sum()
    yield "norm", (x, h, gate, w), lambda: sum(y.square().sum() for y in prn.block_norm_apply(
        h, x, gate=gate, w_post=w, w_pre=w, alpha=w))
    yield "norm before", (h, w), lambda: prn.block_norm_apply(h, w_pre=w)[1].square().sum()
    # a gradient that arrives without a graph of its own
    yield "loss", (x, table), lambda: prn.vocab_loss_apply(x, table, ids)[0].sum()
    yield "lse", (x, table), lambda: prn.vocab_loss_apply(x, table, ids)[1].square().sum()


def test_a_second_derivative_raises():
    """It would lack the operators' parts of it without a sign; the first derivatives are the same either way."""
    for name, leaves, loss in _losses():
        plain = torch.autograd.grad(loss(), leaves)
        total = loss()
        grads = torch.autograd.grad(total, leaves, create_graph=True)
        assert all(torch.equal(a, b) for a, b in zip(plain, grads)), name
        with pytest.raises(RuntimeError, match="first derivatives only"):
            (total + sum(g.square().sum() for g in grads)).backward()
        # gradients that are only kept
        loss().backward(create_graph=True)
        for p, g in zip(leaves, plain):
            with torch.no_grad():
                p.grad.mul_(0.5)
            assert torch.equal(p.grad, 0.5 * g), name
            p.grad = None
