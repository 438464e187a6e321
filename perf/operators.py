"""Cases of the token-model operators: the embedding lookup and its gradient,
the norms at a block boundary with their gate and residual scale, and the
softmax cross entropy over a vocabulary with its gradients.

``run`` computes a case either with this package's operators (``own``) or in
plain form: elementary torch operations in fp32, each result rounded once to
its storage type.  ``exact`` computes the same outputs from the definitions in
float64.

A case is a dict: ``op`` ("embed" | "norm" | "loss"), ``dtype`` ("bf16" |
"f32", the storage type), ``train`` (forward and backward, else the forward
alone) and the sizes: ``N`` tokens, ``d`` channels, ``V`` vocabulary entries.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
IGNORE = -100

# the most work a drawn case may have: the largest listed case of its operator
MOST_EMBED = 262144 * 512
MOST_NORM = 262144 * 512
MOST_LOSS = 32768 * 32768 * 512


def listed():
    return [
        # one token of each of 64 serving slots
        {"name": "embed step", "op": "embed", "dtype": "bf16", "train": False, "N": 64, "d": 512, "V": 32768},
        # a training batch of 8 x 4096 tokens
        {"name": "embed train", "op": "embed", "dtype": "bf16", "train": True, "N": 32768, "d": 512, "V": 32768},
        # a small fp32 model whose sizes are multiples of nothing
        {"name": "embed odd", "op": "embed", "dtype": "f32", "train": True, "N": 4099, "d": 250, "V": 50021},
        # 16 x 16384 tokens over a large vocabulary
        {"name": "embed large", "op": "embed", "dtype": "bf16", "train": True, "N": 262144, "d": 512, "V": 131072},
        # the whole block boundary for one token of 64 serving slots
        {"name": "norm step", "op": "norm", "dtype": "bf16", "train": False, "N": 64, "d": 512,
         "gate": True, "post": True, "res": True, "alpha": True, "pre": True, "act": "silu"},
        # the norm before the first block, 8 x 4096 tokens
        {"name": "norm before", "op": "norm", "dtype": "f32", "train": True, "N": 32768, "d": 256,
         "gate": False, "post": False, "res": False, "alpha": False, "pre": True, "act": "silu"},
        # after the last block of a model with an odd width: no norm follows
        {"name": "norm after odd", "op": "norm", "dtype": "bf16", "train": True, "N": 4097, "d": 1001,
         "gate": True, "post": True, "res": True, "alpha": True, "pre": False, "act": "sigmoid"},
        # the whole boundary, 16 x 16384 tokens
        {"name": "norm boundary", "op": "norm", "dtype": "bf16", "train": True, "N": 262144, "d": 512,
         "gate": True, "post": True, "res": True, "alpha": True, "pre": True, "act": "silu"},
        # the log probabilities of one token of each of 64 slots
        {"name": "loss score", "op": "loss", "dtype": "bf16", "train": False, "N": 64, "d": 512, "V": 32768, "dlse": False},
        # a training step of a small fp32 model
        {"name": "loss fp32", "op": "loss", "dtype": "f32", "train": True, "N": 4096, "d": 256, "V": 32000, "dlse": False},
        # a ragged pack, odd sizes, with the gradient of a penalty on the log partition sum
        {"name": "loss odd", "op": "loss", "dtype": "bf16", "train": True, "N": 5003, "d": 520, "V": 50021, "dlse": True},
        # a training batch of 8 x 4096 tokens
        {"name": "loss train", "op": "loss", "dtype": "bf16", "train": True, "N": 32768, "d": 512, "V": 32768, "dlse": False},
    ]


def _log_int(rng, lo, hi):
    """An integer in [lo, hi], spread over its logarithm; about half of them multiples of 8."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and n >= 8:
        n -= n % 8
    return min(max(n, lo), hi)


def draw(rng):
    op = rng.choice(["embed", "norm", "loss"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "train": rng.random() < 0.7}
    if op == "embed":
        c["d"] = _log_int(rng, 16, 1024)
        c["V"] = _log_int(rng, 256, 131072)
        c["N"] = _log_int(rng, 1, min(262144, MOST_EMBED // c["d"]))
    elif op == "norm":
        c["d"] = _log_int(rng, 16, 8192)
        c["N"] = _log_int(rng, 1, min(262144, MOST_NORM // c["d"]))
        c.update({k: rng.random() < 0.7 for k in ("gate", "post", "res", "alpha")})
        c["pre"] = rng.random() < 0.7 or not (c["gate"] or c["post"] or c["res"] or c["alpha"])
        c["act"] = rng.choice(["silu", "sigmoid"])
    else:
        c["d"] = _log_int(rng, 16, 1024)
        c["V"] = _log_int(rng, 100, 131072)
        most = MOST_LOSS // (c["d"] * c["V"]) // (8 if c["dtype"] == "f32" else 1)
        c["N"] = _log_int(rng, 1, max(1, min(32768, most)))
        c["dlse"] = rng.random() < 0.3
    return c


def _tokens(g, N, V):
    """Token ids whose frequency falls as one over their rank, the ranks spread over the ids."""
    u = torch.rand(N, generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
    return torch.randperm(V, generator=g, device="cuda")[rank]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    N, d = case["N"], case["d"]

    def randn(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    s = dict(case)
    if case["op"] == "embed":
        V = case["V"]
        s["tokens"] = _tokens(g, N, V)
        s["pad_id"] = 0
        s["scale"] = math.sqrt(d)
        s["table"] = randn(V, d, scale=d ** -0.5).to(dt)
        s["dout"] = randn(N, d, scale=0.01).to(dt) if case["train"] else None
    elif case["op"] == "norm":
        s["h"] = randn(N, d, scale=0.5).to(dt)
        s["x"] = randn(N, d, scale=2.0).to(dt) if case["res"] else None
        s["gate_in"] = randn(N, d).to(dt) if case["gate"] else None
        s["w_post"] = 1.0 + randn(d, scale=0.2) if case["post"] else None
        s["w_pre"] = 1.0 + randn(d, scale=0.2) if case["pre"] else None
        s["alpha_w"] = 0.3 + randn(d, scale=0.1) if case["alpha"] else None
        s["dr"] = randn(N, d, scale=0.01).to(dt) if case["train"] else None
        s["dn"] = randn(N, d, scale=0.01).to(dt) if case["train"] and case["pre"] else None
    else:
        V = case["V"]
        W = randn(V, d, scale=d ** -0.5)
        t = _tokens(g, N, V)
        # hidden states of unit size that lean towards their target, so that targets get real probability
        s["x"] = (randn(N, d) + W[t] * (8.0 * torch.rand(N, 1, generator=g, device="cuda"))).to(dt)
        s["W"] = W.to(dt)
        t[torch.rand(N, generator=g, device="cuda") < 0.05] = IGNORE
        s["targets"] = t
        s["scale"] = 1.0
        if case["train"]:
            s["dloss"] = torch.ones(N, device="cuda") / max(1, N)   # the gradient of a mean
            # that of a small multiple of lse^2
            s["dlse"] = randn(N).abs() * (2e-3 / max(1, N)) if case["dlse"] else None
    return s


# ------------------------------------------------------------------ this package's operators ---

def _run_own(s):
    import nonlinear_rnn_amd as prn

    if s["op"] == "embed":
        out = prn.embed(s["tokens"], s["table"], scale=s["scale"], pad_id=s["pad_id"])
        if not s["train"]:
            return {"out": out}
        return {"out": out, "dtable": prn.embed_backward(s["dout"], s["tokens"], s["V"], scale=s["scale"],
                                                         pad_id=s["pad_id"])}
    if s["op"] == "norm":
        kw = dict(gate=s["gate_in"], w_post=s["w_post"], w_pre=s["w_pre"], alpha=s["alpha_w"], act=s["act"], eps=EPS)
        r, n = prn.block_norm(s["h"], s["x"], **kw)
        if not s["train"]:
            return {"r": r, "n": n}
        dh, dx, dgate, dw_post, dw_pre, dalpha = prn.block_norm_backward(s["dr"], s["dn"], s["h"], s["x"], **kw)
        return {"r": r, "n": n, "dh": dh, "dx": dx, "dgate": dgate, "dw_post": dw_post, "dw_pre": dw_pre,
                "dalpha": dalpha}
    loss, lse = prn.vocab_loss(s["x"], s["W"], s["targets"], scale=s["scale"], ignore_index=IGNORE)
    if not s["train"]:
        return {"loss": loss, "lse": lse}
    dx, dW = prn.vocab_loss_backward(s["dloss"], s["x"], s["W"], s["targets"], lse, dlse=s["dlse"], scale=s["scale"],
                                     ignore_index=IGNORE)
    return {"loss": loss, "lse": lse, "dx": dx, "dW": dW}


# ------------------------------------------------------------------ plain forms ---

def _plain_embed(s):
    table, tokens = s["table"], s["tokens"]
    live = tokens != s["pad_id"]
    rows = table[tokens].float() * s["scale"]
    out = torch.where(live[:, None], rows, torch.zeros_like(rows)).to(table.dtype)
    if not s["train"]:
        return {"out": out}
    add = torch.where(live[:, None], s["dout"].float(), torch.zeros_like(rows))
    dtable = torch.zeros(s["V"], s["d"], device=table.device).index_add_(0, tokens, add) * s["scale"]
    return {"out": out, "dtable": dtable.to(table.dtype)}


def _plain_norm(s):
    dt = s["h"].dtype
    h = s["h"].float()
    d = h.shape[-1]
    rstd_h = 1.0 / torch.sqrt((h * h).sum(-1, keepdim=True) / d + EPS)
    hn = h * rstd_h
    u = hn * s["w_post"] if s["post"] else h
    if s["gate"]:
        g = s["gate_in"].float()
        sig = 1.0 / (1.0 + torch.exp(-g))
        a = g * sig if s["act"] == "silu" else sig
        v = u * a
    else:
        v = u
    r = s["alpha_w"] * v if s["alpha"] else v
    if s["res"]:
        r = s["x"].float() + r
    out = {"r": r.to(dt)}
    if s["pre"]:
        rstd_r = 1.0 / torch.sqrt((r * r).sum(-1, keepdim=True) / d + EPS)
        rn = r * rstd_r
        out["n"] = (rn * s["w_pre"]).to(dt)
    if not s["train"]:
        return out
    dr = s["dr"].float()
    if s["pre"]:
        dn = s["dn"].float()
        q = dn * s["w_pre"]
        dr = dr + rstd_r * (q - rn * ((q * rn).sum(-1, keepdim=True) / d))
        out["dw_pre"] = (dn * rn).sum(0)
    dv = dr * s["alpha_w"] if s["alpha"] else dr
    if s["alpha"]:
        out["dalpha"] = (dr * v).sum(0)
    if s["gate"]:
        da = sig * (1.0 + g * (1.0 - sig)) if s["act"] == "silu" else sig * (1.0 - sig)
        out["dgate"] = (dv * u * da).to(dt)
        du = dv * a
    else:
        du = dv
    if s["post"]:
        out["dw_post"] = (du * hn).sum(0)
        q = du * s["w_post"]
        du = rstd_h * (q - hn * ((q * hn).sum(-1, keepdim=True) / d))
    out["dh"] = du.to(dt)
    if s["res"]:
        out["dx"] = dr.to(dt)
    return out


def _plain_loss(s):
    x, W, t = s["x"].float(), s["W"].float(), s["targets"]
    live = t != IGNORE
    at = torch.where(live, t, torch.zeros_like(t))[:, None]
    z = torch.matmul(x, W.t()) * s["scale"]
    m = z.max(-1, keepdim=True).values
    lse = (torch.log(torch.exp(z - m).sum(-1, keepdim=True)) + m)[:, 0]
    loss = torch.where(live, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    if not s["train"]:
        return {"loss": loss, "lse": lse}
    dloss = torch.where(live, s["dloss"], torch.zeros_like(lse))
    dlse = dloss if s["dlse"] is None else dloss + s["dlse"]
    dz = torch.exp(z - lse[:, None]) * dlse[:, None]
    dz.scatter_add_(1, at, -dloss[:, None])
    dz *= s["scale"]
    return {"loss": loss, "lse": lse, "dx": torch.matmul(dz, W).to(s["x"].dtype),
            "dW": torch.matmul(dz.t(), x).to(s["W"].dtype)}


def run(state):
    if own:
        return _run_own(state)
    return {"embed": _plain_embed, "norm": _plain_norm, "loss": _plain_loss}[state["op"]](state)


# ------------------------------------------------------------------ work and exact values ---

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    N, d, train = case["N"], case["d"], case["train"]
    if case["op"] == "embed":
        # each distinct row once; with these frequencies about V (1 - E[(1 - p)^N]) of them
        V = case["V"]
        ln = math.log(V + 1.0)
        p = [math.log1p(1.0 / (k + 1.0)) / ln for k in range(V)]
        rows = sum(1.0 - math.exp(N * math.log1p(-q)) for q in p)
        b = 8 * N + rows * d * e + N * d * e
        f = N * d
        if train:
            b += N * d * e + V * d * e
            f += N * d + rows * d
        return {"bytes": b, "flops": f}
    if case["op"] == "norm":
        arrays = 1 + case["gate"] + case["res"]
        b = (arrays + 1 + case["pre"]) * N * d * e + (case["post"] + case["pre"] + case["alpha"]) * 4 * d
        f = N * d * (1 + 4 * case["post"] + 8 * case["gate"] + case["res"] + case["alpha"] + 4 * case["pre"])
        if train:
            # the operands are there already: the output gradients in, the input gradients out
            b += (1 + case["pre"] + arrays) * N * d * e + (case["post"] + case["pre"] + case["alpha"]) * 4 * d
            f += N * d * (1 + 8 * case["post"] + 8 * case["gate"] + 3 * case["alpha"] + 8 * case["pre"])
        return {"bytes": b, "flops": f}
    V = case["V"]
    b = (N + V) * d * e + 16 * N
    f = 2.0 * N * V * d
    if train:
        b += (N + V) * d * e + 4 * N * (1 + case["dlse"])
        f += 4.0 * N * V * d
    return {"bytes": b, "flops": f}


def _exact_embed(s):
    tokens, table = s["tokens"], s["table"].double()
    keep = (tokens != s["pad_id"]).double().unsqueeze(1)
    out = {"out": table.index_select(0, tokens) * keep * s["scale"]}
    if s["train"]:
        order = torch.argsort(tokens, stable=True)
        rows = (s["dout"].double() * keep * s["scale"]).index_select(0, order)
        grad = torch.zeros(s["V"], s["d"], dtype=torch.float64, device=rows.device)
        out["dtable"] = grad.index_put_((tokens.index_select(0, order),), rows, accumulate=True)
    return out


def _exact_norm(s):
    def leaf(v):
        return None if v is None else v.double().requires_grad_()

    h, x, g, wo, wi, al = (leaf(s[k]) for k in ("h", "x", "gate_in", "w_post", "w_pre", "alpha_w"))
    with torch.enable_grad():
        v = h if wo is None else h * torch.pow(h.pow(2).mean(-1, keepdim=True) + EPS, -0.5) * wo
        if g is not None:
            v = v * (torch.sigmoid(g) * (g if s["act"] == "silu" else 1.0))
        r = v if al is None else v * al
        r = r if x is None else r + x
        outs = {"r": r}
        if wi is not None:
            outs["n"] = r * torch.pow(r.pow(2).mean(-1, keepdim=True) + EPS, -0.5) * wi
        if s["train"]:
            names = [(n, v) for n, v in (("dh", h), ("dx", x), ("dgate", g), ("dw_post", wo), ("dw_pre", wi),
                                         ("dalpha", al)) if v is not None]
            total = (r * s["dr"].double()).sum()
            if wi is not None:
                total = total + (outs["n"] * s["dn"].double()).sum()
            grads = torch.autograd.grad(total, [v for _, v in names])
            outs.update({n: v for (n, _), v in zip(names, grads)})
    return {k: v.detach() for k, v in outs.items()}


def _exact_loss(s):
    # rows in pieces, so that float64 logits of the largest case fit
    N, V = s["N"], s["V"]
    W = s["W"].double()
    piece = max(1, min(N, (1 << 29) // V))
    loss, lse, dxs, dW = [], [], [], torch.zeros_like(W)
    for lo in range(0, N, piece):
        x, t = s["x"][lo:lo + piece].double(), s["targets"][lo:lo + piece]
        live = t >= 0
        z = (x @ W.T).mul_(s["scale"])
        L = torch.logsumexp(z, 1)
        rows = torch.arange(x.shape[0], device=x.device)[live]
        losses = torch.zeros_like(L)
        losses[live] = L[live] - z[rows, t[live]]
        loss.append(losses)
        lse.append(L)
        if s["train"]:
            dl = s["dloss"][lo:lo + piece].double() * live
            p = z.sub_(L[:, None]).exp_()
            p.mul_((dl if s["dlse"] is None else dl + s["dlse"][lo:lo + piece].double())[:, None])
            p[rows, t[live]] -= dl[live]
            p.mul_(s["scale"])
            dxs.append(p @ W)
            dW += p.T @ x
    out = {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    if s["train"]:
        out.update(dx=torch.cat(dxs), dW=dW)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"embed": _exact_embed, "norm": _exact_norm, "loss": _exact_loss}[s["op"]](s)
