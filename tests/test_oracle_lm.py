"""CPU pins of oracle.lm: gradients against central differences, every part of
the block boundary on and off, and special cases with known answers."""
import itertools

import numpy as np
import pytest

from oracle import lm


def _diff(f, y, dy, eps=1e-6):
    return (f(y + eps * dy) - f(y - eps * dy)) / (2 * eps)


def test_embed_gradient_is_the_transpose_of_the_lookup():
    rng = np.random.default_rng(0)
    tokens = np.array([3, 0, 3, 9, -1, 2, 3])
    table, dout = rng.standard_normal((5, 4)), rng.standard_normal((7, 4))
    out = lm.embed(tokens, table, 1.5, pad_id=0)
    assert np.isnan(out[[3, 4]]).all() and (out[1] == 0).all()
    grad, _, count = lm.embed_backward(dout, tokens, 5, 1.5, pad_id=0)
    assert count.tolist() == [0, 0, 1, 3, 0]
    live = [0, 2, 5, 6]
    assert np.isclose((out[live] * dout[live]).sum(), (grad * table).sum())


@pytest.mark.parametrize("gate,post,pre,alpha,res", itertools.product([False, True], repeat=5))
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_block_norm_gradients_against_differences(gate, post, pre, alpha, res, act):
    rng = np.random.default_rng(1)
    N, d = 3, 7
    draw = lambda on, *s: rng.standard_normal(s) if on else None   # noqa: E731
    kw = dict(h=draw(True, N, d), x=draw(res, N, d), gate=draw(gate, N, d), w_post=draw(post, d),
              w_pre=draw(pre, d), alpha=draw(alpha, d))
    dr, dn = rng.standard_normal((N, d)), draw(pre, N, d)

    def total(**k):
        r, n = lm.block_norm(**k, act=act, eps=1e-3)
        return (r * dr).sum() + (0.0 if n is None else (n * dn).sum())

    got = lm.block_norm_backward(dr, dn, **kw, act=act, eps=1e-3)
    for name in kw:
        if kw[name] is None:
            assert "d" + name not in got
            continue
        dy = rng.standard_normal(kw[name].shape)
        want = _diff(lambda y: total(**{**kw, name: y}), kw[name], dy)
        assert abs((got["d" + name] * dy).sum() - want) < 1e-7 * max(1.0, abs(want))
    size = lm.block_norm_backward(dr, dn, **kw, act=act, eps=1e-3, size=True)
    for k in got:
        assert (size[k] >= np.abs(got[k]) * (1 - 1e-12)).all()


def test_vocab_loss_gradients_against_differences_and_special_rows():
    rng = np.random.default_rng(2)
    N, V, d = 4, 6, 3
    x, W = rng.standard_normal((N, d)), rng.standard_normal((V, d))
    t = np.array([1, -100, 5, 0])
    dloss, dlse = rng.standard_normal(N), rng.standard_normal(N)

    def total(x, W):
        loss, lse, _ = lm.vocab_loss(x, W, t, 0.7)
        return (loss * dloss).sum() + (lse * dlse).sum()

    loss, lse, z = lm.vocab_loss(x, W, t, 0.7)
    assert loss[1] == 0.0 and np.allclose(np.exp(z - lse[:, None]).sum(1), 1.0)
    dz = lm.vocab_loss_dz(dloss, dlse, z, lse, t, 0.7)
    for y, g, f in ((x, dz @ W, lambda y: total(y, W)), (W, dz.T @ x, lambda y: total(x, y))):
        dy = rng.standard_normal(y.shape)
        assert abs((g * dy).sum() - _diff(f, y, dy)) < 1e-8
    assert np.isnan(lm.vocab_loss(x, W, np.array([6, 0, 0, -1]))[0][[0, 3]]).all()
    # one entry: certain
    assert np.allclose(lm.vocab_loss(x, W[:1], np.zeros(N, dtype=int))[0], 0.0)
