"""A token model on the recurrence, from ids to loss and back, and its serving step.

    x = embed(tokens)                                         token ids to rows
    for every layer:
        x, n = block_norm(h, x, gate, w_post, alpha, w_pre)   the seam before the layer
        h    = newton(input_proj(n))                          the recurrence
        gate = n Wg^T
    y = block_norm(h, x, ...) and the last norm               the seam after the last layer
    loss, lse = vocab_loss(y, E, targets)                     against the embedding table itself

The table is shared by the lookup and the loss, so its gradient is the sum of
both.  Serving runs the same weights one token at a time: the same seams, the
fused decode step on a carry per slot, and the same loss for scoring.

With --linear the blocks are of a gated linear recurrence, which is one scan and
no Newton iteration, each with a feed-forward half and dropout:

        x, m = block_norm(h, x, gate, w_post, alpha, w_ffn)   h = gated_scan(input_proj(n))
        x    = x + dropout(gated_ffn(m) Wd^T)

    python examples/token_model.py                 a minute of training on synthetic tokens, then scoring
    python examples/token_model.py --dtype bf16 --width 512 --vocab 32768 --batch 8 --length 4096
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nonlinear_rnn_amd as prn  # noqa: E402
from nonlinear_rnn_amd import binding  # noqa: E402


class TokenModel(torch.nn.Module):
    """`layers` gated GRU blocks of `width` channels over a vocabulary of V tokens; id V - 1 pads."""

    def __init__(self, V, width, layers, dtype=torch.float32):
        super().__init__()
        def new(*shape, scale=1.0, kind=dtype):
            return torch.nn.Parameter((torch.randn(*shape, device="cuda") * scale).to(kind))
        f32 = torch.float32
        self.V, self.width, self.pad = V, width, V - 1
        self.table = new(V, width, scale=width ** -0.5)
        self.layers = torch.nn.ModuleList()
        for _ in range(layers):
            layer = torch.nn.Module()
            layer.W = new(3 * width, width, scale=width ** -0.5)
            layer.Wg = new(width, width, scale=width ** -0.5)
            layer.bias = torch.nn.Parameter(torch.zeros(3 * width, device="cuda"))
            layer.a = torch.nn.Parameter(torch.rand(3, width, device="cuda") - 0.5)
            layer.w_pre, layer.w_post = (torch.nn.Parameter(torch.ones(width, device="cuda")) for _ in range(2))
            layer.alpha = new(width, scale=0.1, kind=f32)
            self.layers.append(layer)
        self.w_out = torch.nn.Parameter(torch.ones(width, device="cuda"))

    def _seams(self):
        """(weights of the block that ends, w_pre of the one that begins) in order."""
        blocks = [None, *self.layers]
        return [(done, self.layers[i].w_pre if i < len(self.layers) else self.w_out) for i, done in enumerate(blocks)]

    def _seam(self, done, w_pre, h, x, gate):
        if done is None:   # before the first block there is only the norm
            return prn.block_norm_apply(x, w_pre=w_pre)
        return prn.block_norm_apply(h, x, gate=gate, w_post=done.w_post, alpha=done.alpha, w_pre=w_pre)

    def features(self, tokens, K=None):
        """(B, T) ids -> (B, T, width): the rows that meet the table's in the loss."""
        x = prn.embed_apply(tokens, self.table, scale=self.width ** 0.5, pad_id=self.pad)
        h = gate = None
        for i, (done, w_pre) in enumerate(self._seams()):
            x, n = self._seam(done, w_pre, h, x, gate)
            if i < len(self.layers):
                layer = self.layers[i]
                gate = torch.nn.functional.linear(n, layer.Wg)
                h = prn.newton_apply(prn.input_proj_apply(n, layer.W, layer.bias, cell="gru"), layer.a, K, cell="gru")
        return n

    def loss(self, tokens, targets, K=None, z_loss=0.0):
        """Mean cross entropy over the targets that are not padding, and z_loss times the mean squared log
        partition sum."""
        loss, lse = prn.vocab_loss_apply(self.features(tokens, K), self.table, targets, ignore_index=self.pad)
        live = (targets != self.pad).sum().clamp(min=1)
        total = loss.sum() / live
        return total + z_loss * (lse * lse).mean() if z_loss else total

    @torch.no_grad()
    def step(self, tokens, carry, targets):
        """One token of every slot: (B) ids, the carry of an earlier step or None, the ids to score next.
        Returns (log probabilities of targets, the next carry)."""
        x = prn.embed(tokens, self.table, scale=self.width ** 0.5, pad_id=self.pad)
        h = gate = None
        new = []
        for i, (done, w_pre) in enumerate(self._seams()):
            x, n = self._seam(done, w_pre, h, x, gate)
            if i < len(self.layers):
                layer = self.layers[i]
                gate = torch.nn.functional.linear(n, layer.Wg)
                state = n.new_empty((len(tokens), 1, self.width))
                binding.prn_decode_step(n, layer.W, layer.bias, layer.a, state, cell="gru",
                                        state_in=None if carry is None else carry[i])
                new.append(state)
                h = state[:, 0]
        loss, _ = prn.vocab_loss(n, self.table, targets, ignore_index=self.pad)
        return -loss, new


class LinearTokenModel(torch.nn.Module):
    """`layers` blocks of a gated linear recurrence (cell "glr" or "glri") of `width` channels and a gated feed-forward
    product of `hidden`, dropout of a share p before every feed-forward half joins the stream; id V - 1 pads."""

    def __init__(self, V, width, layers, hidden, p=0.0, cell="glr", dtype=torch.float32):
        super().__init__()
        def new(*shape, scale=1.0, kind=dtype):
            return torch.nn.Parameter((torch.randn(*shape, device="cuda") * scale).to(kind))
        self.V, self.width, self.pad, self.p, self.cell = V, width, V - 1, p, cell
        self.table = new(V, width, scale=width ** -0.5)
        self.layers = torch.nn.ModuleList()
        gates = binding.GATES[cell]
        for _ in range(layers):
            layer = torch.nn.Module()
            layer.W = new(gates * width, width, scale=width ** -0.5)
            bias = torch.zeros(gates * width, device="cuda")
            bias[:width] = torch.linspace(0.0, 6.0, width, device="cuda")   # memories of a few steps to hundreds
            layer.bias = torch.nn.Parameter(bias)
            layer.Wg = new(width, width, scale=width ** -0.5)
            layer.Wf = new(2 * hidden, width, scale=width ** -0.5)
            layer.Wd = new(width, hidden, scale=0.3 * hidden ** -0.5)
            layer.w_pre, layer.w_post, layer.w_ffn = (torch.nn.Parameter(torch.ones(width, device="cuda")) for _ in range(3))
            layer.alpha = new(width, scale=0.3, kind=torch.float32)
            self.layers.append(layer)
        self.w_out = torch.nn.Parameter(torch.ones(width, device="cuda"))
        self.register_buffer("waits", torch.zeros(1, dtype=torch.int32, device="cuda"), persistent=False)

    def _block(self, layer, x, h, n, seed, offset):
        """The rest of a block after its recurrence: the stream x behind it."""
        gate = torch.nn.functional.linear(n, layer.Wg)
        x, m = prn.block_norm_apply(h, x, gate=gate, w_post=layer.w_post, alpha=layer.alpha, w_pre=layer.w_ffn)
        y = torch.nn.functional.linear(prn.gated_ffn_apply(m, layer.Wf), layer.Wd)
        return prn.dropout_apply(y, 0.0 if seed is None else self.p, seed=seed or 0, offset=offset, residual=x)

    def features(self, tokens, seed=None, step=0, cu_seqlens=None):
        """(B, T) ids -> (B, T, width); with a seed dropout is on, its numbers those of (seed, step, layer)."""
        x = prn.embed_apply(tokens, self.table, scale=self.width ** 0.5, pad_id=self.pad)
        for i, layer in enumerate(self.layers):
            _, n = prn.block_norm_apply(x, w_pre=layer.w_pre)
            h = prn.gated_scan_apply(prn.input_proj_apply(n, layer.W, layer.bias, cell=self.cell), cell=self.cell,
                                     cu_seqlens=cu_seqlens, error_out=self.waits)
            x = self._block(layer, x, h, n, seed, step * len(self.layers) + i)
        return prn.block_norm_apply(x, w_pre=self.w_out)[1]

    def loss(self, tokens, targets, z_loss=0.0, seed=None, step=0):
        """Mean cross entropy over the targets that are not padding."""
        loss, lse = prn.vocab_loss_apply(self.features(tokens, seed, step), self.table, targets, ignore_index=self.pad)
        total = loss.sum() / (targets != self.pad).sum().clamp(min=1)
        return total + z_loss * (lse * lse).mean() if z_loss else total

    @torch.no_grad()
    def step(self, tokens, carry, targets):
        """As TokenModel.step: one token of every slot."""
        x = prn.embed(tokens, self.table, scale=self.width ** 0.5, pad_id=self.pad)
        new = []
        for i, layer in enumerate(self.layers):
            _, n = prn.block_norm(x, w_pre=layer.w_pre)
            state = n.new_empty((len(tokens), 1, self.width))
            binding.prn_decode_step(n, layer.W, layer.bias, None, state, cell=self.cell,
                                    state_in=None if carry is None else carry[i])
            new.append(state)
            x = self._block(layer, x, state[:, 0], n, None, 0)
        loss, _ = prn.vocab_loss(prn.block_norm(x, w_pre=self.w_out)[1], self.table, targets, ignore_index=self.pad)
        return -loss, new


def chain(B, T, V, generator, follow=0.9):
    """Synthetic ids: a token is mostly followed by a fixed other one, so there is something to learn.
    (inputs, targets), both (B, T), the last position of every row padded."""
    after = torch.randperm(V - 1, generator=generator, device="cuda")
    noise = torch.randint(V - 1, (B, T + 1), generator=generator, device="cuda")
    keep = torch.rand(B, T + 1, generator=generator, device="cuda") < follow
    ids = noise.clone()
    for t in range(1, T + 1):
        ids[:, t] = torch.where(keep[:, t], after[ids[:, t - 1]], noise[:, t])
    targets = ids[:, 1:].clone()
    targets[:, -1] = V - 1
    return ids[:, :-1].contiguous(), targets


def train(model, tokens, targets, steps, lr=3e-3, log=None, seed=None):
    """Plain Adam on one batch; the losses.  seed: that of a model's dropout."""
    optimizer = torch.optim.Adam(model.parameters(), lr=lr)
    losses = []
    for i in range(steps):
        optimizer.zero_grad(set_to_none=True)
        loss = model.loss(tokens, targets, z_loss=1e-4, **({} if seed is None else dict(seed=seed, step=i)))
        loss.backward()
        losses.append(loss.item())
        if isinstance(model, LinearTokenModel):
            prn.check_waits(model.waits)   # a wait that gave up has left NaN (newton_apply raises by itself)
        optimizer.step()
        if log and (i % 5 == 0 or i == steps - 1):
            log(f"step {i:3d}  loss {losses[-1]:.4f}")
    return losses


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--vocab", type=int, default=2000)
    p.add_argument("--width", type=int, default=256)
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--length", type=int, default=512)
    p.add_argument("--steps", type=int, default=40)
    p.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    p.add_argument("--linear", action="store_true", help="blocks of a gated linear recurrence with feed-forward halves")
    p.add_argument("--dropout", type=float, default=0.1, help="of the linear model")
    args = p.parse_args()
    torch.manual_seed(0)
    g = torch.Generator(device="cuda").manual_seed(0)
    dtype = torch.bfloat16 if args.dtype == "bf16" else torch.float32
    model = (LinearTokenModel(args.vocab, args.width, args.layers, 11 * args.width // 4, args.dropout, dtype=dtype)
             if args.linear else TokenModel(args.vocab, args.width, args.layers, dtype))
    seed = 1 if args.linear else None
    tokens, targets = chain(args.batch, args.length, args.vocab, g)

    def say(text):
        print(text, flush=True)
    train(model, tokens, targets, 1, seed=seed)   # the first call loads the library
    torch.cuda.synchronize()
    start = time.perf_counter()
    losses = train(model, tokens, targets, args.steps, log=say, seed=seed)
    torch.cuda.synchronize()
    took = (time.perf_counter() - start) / args.steps
    say(f"{args.steps} steps, {took * 1e3:.2f} ms each, {tokens.numel() / took / 1e6:.2f} M tokens/s; "
        f"loss {losses[0]:.3f} -> {losses[-1]:.3f}")

    carry, total = None, torch.zeros(args.batch, device="cuda")
    slots = min(args.length, 32)
    for t in range(slots):
        score, carry = model.step(tokens[:, t].contiguous(), carry, targets[:, t].contiguous())
        total += score
    say(f"served {slots} tokens in {args.batch} slots: mean log probability {(total / slots).mean().item():.3f}")


if __name__ == "__main__":
    main()
