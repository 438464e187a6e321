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


def train(model, tokens, targets, steps, lr=3e-3, log=None):
    """Plain Adam on one batch; the losses."""
    optimizer = torch.optim.Adam(model.parameters(), lr=lr)
    losses = []
    for i in range(steps):
        optimizer.zero_grad(set_to_none=True)
        loss = model.loss(tokens, targets, z_loss=1e-4)
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
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
    args = p.parse_args()
    torch.manual_seed(0)
    g = torch.Generator(device="cuda").manual_seed(0)
    model = TokenModel(args.vocab, args.width, args.layers, torch.bfloat16 if args.dtype == "bf16" else torch.float32)
    tokens, targets = chain(args.batch, args.length, args.vocab, g)

    def say(text):
        print(text, flush=True)
    train(model, tokens, targets, 1)   # the first call loads the library
    torch.cuda.synchronize()
    start = time.perf_counter()
    losses = train(model, tokens, targets, args.steps, log=say)
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
