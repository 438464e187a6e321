"""CPU pins of oracle.gated: gradients against central differences, sequences
of a pack against each alone, the generator against its published vectors."""
import numpy as np
import pytest

from oracle import gated

G = {"glr": 2, "glri": 3}


def _diff(f, y, dy, eps=1e-6):
    return (f(y + eps * dy) - f(y - eps * dy)) / (2 * eps)


@pytest.mark.parametrize("cell", ["glr", "glri"])
@pytest.mark.parametrize("ragged", [False, True])
def test_scan_gradients_against_differences(cell, ragged):
    rng = np.random.default_rng(0)
    B, T, d = (1, 11, 3) if ragged else (2, 7, 3)
    cu = np.array([0, 4, 4, 9, 11]) if ragged else None
    rows = 4 if ragged else B
    x, h0 = rng.standard_normal((B, T, G[cell], d)), rng.standard_normal((rows, 1, d))
    dH, dlast = rng.standard_normal((B, T, d)), rng.standard_normal((rows, 1, d))

    def total(x, h0):
        H, last = gated.gated_scan(cell, x, h0, cu)
        return (H * dH).sum() + (last * dlast).sum()

    dx, dh0 = gated.gated_scan_backward(cell, x, dH, h0, cu, dlast)
    for _ in range(3):
        r, s = rng.standard_normal(x.shape), rng.standard_normal(h0.shape)
        assert np.isclose((dx * r).sum(), _diff(lambda y: total(y, h0), x, r), rtol=1e-7, atol=1e-9)
        assert np.isclose((dh0 * s).sum(), _diff(lambda y: total(x, y), h0, s), rtol=1e-7, atol=1e-9)


def test_a_pack_is_its_sequences_and_an_empty_one_keeps_its_state():
    rng = np.random.default_rng(1)
    x, h0 = rng.standard_normal((1, 9, 2, 4)), rng.standard_normal((4, 1, 4))
    cu = [0, 5, 5, 6, 9]
    H, last = gated.gated_scan("glr", x, h0, cu)
    for j in range(4):
        lo, hi = cu[j], cu[j + 1]
        alone, end = gated.gated_scan("glr", x[:, lo:hi], h0[j:j + 1])
        assert (alone == H[:, lo:hi]).all() and (end[0] == last[j]).all()
    assert (last[1] == h0[1]).all()


def test_a_held_gate_keeps_and_an_open_one_replaces():
    x = np.zeros((1, 3, 2, 1))
    x[0, :, 0, 0], x[0, :, 1, 0] = [-800.0, 800.0, 0.0], [3.0, 5.0, 7.0]
    H, _ = gated.gated_scan("glr", x)
    assert H[0, :, 0].tolist() == [3.0, 3.0, 5.0]


@pytest.mark.parametrize("kind", ["silu", "sigmoid"])
def test_ffn_gradients_against_differences(kind):
    rng = np.random.default_rng(2)
    x, W, dout = rng.standard_normal((4, 5)), rng.standard_normal((6, 5)), rng.standard_normal((4, 3))
    total = lambda x, W: (gated.gated_ffn(x, W, kind) * dout).sum()   # noqa: E731
    dx, dW = gated.gated_ffn_backward(x, W, dout, kind)
    r, s = rng.standard_normal(x.shape), rng.standard_normal(W.shape)
    assert np.isclose((dx * r).sum(), _diff(lambda y: total(y, W), x, r), rtol=1e-7)
    assert np.isclose((dW * s).sum(), _diff(lambda y: total(x, y), W, s), rtol=1e-7)


def test_philox_known_answers():
    """The published test vectors of philox4x32-10: counters and keys of zeros, of ones, and of the digits of pi."""
    m = (1 << 64) - 1
    assert gated.philox([0], 0, 0)[0].tolist() == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert gated.philox([m], m, m)[0].tolist() == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    words = gated.philox([0x85a308d3243f6a88], 0x0370734413198a2e, 0x299f31d0a4093822)[0]
    assert words.tolist() == [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


def test_dropout_keeps_its_share_and_its_mean():
    keep = gated.kept(40000, 0.25, 7, 3)
    assert abs(keep.mean() - 0.75) < 4 * (0.25 * 0.75 / 40000) ** 0.5   # four standard deviations
    assert not gated.kept(100, 1.0, 1, 1).any() and gated.kept(100, 0.0, 1, 1).all()
    x = np.ones(16)
    assert set(gated.dropout(x, 0.5, 5, 0).tolist()) == {0.0, 2.0}
    assert (gated.dropout(np.full(8, np.nan), 1.0, 5, 0, residual=x[:8]) == 1.0).all()
