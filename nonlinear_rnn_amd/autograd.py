"""What the differentiable operators without a second derivative share."""
from __future__ import annotations

import torch


class _FirstDerivatives(torch.autograd.Function):
    """Copies of gradients, and an error where a derivative of theirs is asked for."""

    @staticmethod
    def forward(ctx, count, *tensors):
        return tuple(t.clone() for t in tensors[:count])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the token-model operators have first derivatives only")


def first(grads, *sources):
    """A backward pass's gradients.  Under create_graph they would come without a graph, and a derivative of theirs
    would silently lack this operator's part: it raises instead."""
    sources = [s for s in sources if s is not None and s.requires_grad]
    if not torch.is_grad_enabled() or not sources:
        return grads
    given = [g for g in grads if g is not None]
    tied = iter(_FirstDerivatives.apply(len(given), *given, *sources))
    return tuple(None if g is None else next(tied) for g in grads)
