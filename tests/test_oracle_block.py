"""Pins of the fp64 definitions in oracle/block.py: gradients against central
differences of the forward they belong to, the activations against closed
values, and the dropout generator against its authors' known answers."""
import math

import numpy as np
import pytest

from oracle import block

H = 1e-6


def diff(f, x):
    """Central differences of the scalar f at x."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += H
        b[i] -= H
        g[i] = (f(a) - f(b)) / (2 * H)
    return g


def close(a, b):
    """Central differences of smooth functions of order 1 values: truncation
    H^2 and rounding 2^-52 / H, so 1e-8 with room for sums of a few dozen."""
    return np.allclose(a, b, rtol=1e-6, atol=1e-7)


def test_philox_known_answers():
    """The published vectors of philox4x32 with ten rounds: zeros, ones, and digits of pi."""
    ones = 0xFFFFFFFF
    for c, k, want in [
        ((0,) * 4, (0,) * 2, (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
        ((ones,) * 4, (ones,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
        ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
         (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
    ]:
        assert tuple(int(v) for v in block.philox(c, k)) == want


def test_mask_rate_offsets_rows_and_negative_numbers():
    T, d = 400, 501
    for p in (0.0625, 0.1, 0.5, 0.9):
        keep = block.dropout_keep(T, d, p, 7, 9)
        sd = math.sqrt(p * (1 - p) / keep.size)
        assert abs(keep.mean() - (1 - p)) < 5 * sd
        assert abs(keep.mean(axis=0) - (1 - p)).max() < 6 * math.sqrt(p * (1 - p) / T)
    whole = block.dropout_keep(T, d, 0.3, 7, 9)
    assert np.array_equal(block.dropout_keep(100, d, 0.3, 7, 9, row0=123), whole[123:223])
    assert np.array_equal(block.dropout_keep(T, 37, 0.3, 7, 9), whole[:, :37])
    assert (block.dropout_keep(T, d, 0.3, 7, 10) != whole).mean() > 0.3
    assert (block.dropout_keep(T, d, 0.3, 8, 9) != whole).mean() > 0.3
    # 64-bit patterns: -1 and 2^64 - 1 are the same number
    assert np.array_equal(block.dropout_keep(9, 9, 0.3, -1, -2), block.dropout_keep(9, 9, 0.3, 2 ** 64 - 1, 2 ** 64 - 2))
    assert block.dropout_keep(9, 9, 0.0, 1, 2).all()


@pytest.mark.parametrize("kind", block.ACTS)
def test_activation_slopes(kind):
    z = np.linspace(-6, 6, 241) + 0.003  # no sample at ReLU's corner
    num = (block.act(z + H, kind) - block.act(z - H, kind)) / (2 * H)
    assert close(block.act_slope(z, kind), num)


def test_activation_values():
    assert block.act(np.array([1.0]), "gelu")[0] == pytest.approx(0.8413447460685429, rel=1e-14)
    assert block.act(np.array([1.0]), "silu")[0] == pytest.approx(1 / (1 + math.exp(-1)), rel=1e-14)
    assert block.act(np.array([1.0]), "gelu_tanh")[0] == pytest.approx(0.8411919906082768, rel=1e-12)
    assert abs(block.act(np.linspace(-6, 6, 99), "gelu") - block.act(np.linspace(-6, 6, 99), "gelu_tanh")).max() < 5e-4


def test_layernorm_gradients():
    rng = np.random.default_rng(0)
    x, g, b, c = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=7), rng.normal(size=(3, 7))
    eps = 1e-3
    f = lambda x, g, b: float((block.layernorm_fwd(x, g, b, eps)[0] * c).sum())  # noqa: E731
    _, m, r = block.layernorm_fwd(x, g, b, eps)
    dx, dg, db = block.layernorm_bwd(x, g, m, r, c)
    assert close(dx, diff(lambda v: f(v, g, b), x))
    assert close(dg, diff(lambda v: f(x, v, b), g))
    assert close(db, diff(lambda v: f(x, g, v), b))


@pytest.mark.parametrize("kind", block.ACTS)
@pytest.mark.parametrize("p", [0.0, 0.4])
def test_linear_gradients(kind, p):
    """Two layers with dropout between them: the gradient of the first's
    pre-activation and bias, and the step from the output's own gradient."""
    rng = np.random.default_rng(1)
    A, W1, b1 = rng.normal(size=(4, 5)), rng.normal(size=(6, 5)), rng.normal(size=6)
    W2, c = rng.normal(size=(3, 6)), rng.normal(size=(4, 3))
    keep = block.dropout_keep(4, 6, p, 3, 4)
    f = lambda U: float(((block.drop(block.act(U, kind), p, keep) @ W2.T) * c).sum())  # noqa: E731
    C, U = block.linear_fwd(A, W1, b1, kind, p, keep, R=0.0)
    assert close(C, block.drop(block.act(U, kind), p, keep))
    dZ, db = block.linear_bwd_act(c, W2, U, kind, p, keep)
    assert close(dZ, diff(f, U))
    assert close(db, diff(lambda v: f(A @ W1.T + v), b1))
    assert np.array_equal(block.act_bwd(c @ W2, U, kind, p, keep)[0], dZ)


@pytest.mark.parametrize("kind", block.ACTS)
def test_gated_gradients(kind):
    rng = np.random.default_rng(2)
    x, Wg, Wu = rng.normal(size=(4, 5)), rng.normal(size=(6, 5)), rng.normal(size=(6, 5))
    Wd, c = rng.normal(size=(3, 6)), rng.normal(size=(4, 3))
    f = lambda g, u: float(((block.act(g, kind) * u) @ Wd.T * c).sum())  # noqa: E731
    h, g, u = block.gated_fwd(x, Wg, Wu, kind)
    dg, du, h2 = block.gated_bwd(c, Wd, g, u, kind)
    assert np.array_equal(h, h2)
    assert close(dg, diff(lambda v: f(v, u), g))
    assert close(du, diff(lambda v: f(g, v), u))
