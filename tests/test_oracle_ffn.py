"""The feed-forward operators' oracle against differences of its own forward
pass, invariants and closed forms."""
import math

import numpy as np
import pytest

from oracle import ffn_oracle as O


def differences(f, x, step=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        g[i] = (f(a) - f(b)) / (2 * step)
    return g


def test_layernorm_gradient_against_differences():
    rng = np.random.default_rng(0)
    h, w, b = rng.normal(size=(3, 7)), 1 + 0.2 * rng.normal(size=7), rng.normal(size=7)
    dy, dh = rng.normal(size=(3, 7)), rng.normal(size=(3, 7))
    dx, dw, db = O.layernorm_bwd(dy, h, w, 1e-3, dh)
    f = lambda h_, w_, b_: (O.layernorm(h_, w_, b_, 1e-3)[0] * dy).sum() + (h_ * dh).sum()
    assert np.allclose(dx, differences(lambda v: f(v, w, b), h), atol=1e-8)
    assert np.allclose(dw, differences(lambda v: f(h, v, b), w), atol=1e-8)
    assert np.allclose(db, differences(lambda v: f(h, w, v), b), atol=1e-8)


def test_layernorm_invariants():
    rng = np.random.default_rng(1)
    h = rng.normal(size=(4, 50))
    y, mean, rstd, _ = O.layernorm(h, np.ones(50), None, 0.0)
    assert np.allclose(y.mean(1), 0) and np.allclose(y.var(1), 1)
    again = O.layernorm(3.0 * h + 7.0, np.ones(50), None, 0.0)
    assert np.allclose(again[0], y) and np.allclose(again[1], 3 * mean + 7)
    assert np.allclose(again[2], rstd / 3)
    # its gradient is orthogonal to the ones and to the row itself
    dx = O.layernorm_bwd(rng.normal(size=(4, 50)), h, np.ones(50), 0.0)[0]
    assert np.allclose(dx.sum(1), 0) and np.allclose((dx * h).sum(1), 0)


def test_dropout_mask():
    keep = O.dropout_keep(64, 500, 0.25, 12345, 7)
    assert abs(keep.mean() - 0.75) < 5 * math.sqrt(0.25 * 0.75 / keep.size)
    assert not np.array_equal(keep, O.dropout_keep(64, 500, 0.25, 12345, 8))
    assert not np.array_equal(keep, O.dropout_keep(64, 500, 0.25, 12346, 7))
    # the mask of a larger p drops what the smaller dropped
    assert not (O.dropout_keep(64, 500, 0.5, 12345, 7) & ~keep).any()
    assert np.array_equal(keep[40:], O.dropout_keep(24, 500, 0.25, 12345, 7, row0=40))
    assert O.dropout_keep(3, 9, 0.0, 1, 0).all() and not O.dropout_keep(3, 9, 1.0, 1, 0).any()
    # unbiased, and the residual is only added
    x = np.ones((64, 500), np.float32)
    y = O.dropout(x, 0.25, 12345, 7)
    assert set(np.unique(y)) == {np.float32(0), np.float32(65536 / (65536 - 16384))}
    assert np.array_equal(O.dropout(x, 0.25, 12345, 7, res=2 * x), y + 2)


@pytest.mark.parametrize("kind", [O.SILU, O.GELU])
def test_activations(kind):
    g = np.linspace(-30, 30, 2001)
    value, slope = O.act(g, kind)
    up, down = (O.act(g + d, kind)[0] for d in (1e-6, -1e-6))
    assert np.allclose(slope, (up - down) / 2e-6, atol=1e-8)
    # value(g) - value(-g) = g, for both
    assert np.allclose(value - O.act(-g, kind)[0], g)
    assert np.isclose(O.act(1.0, kind)[0], {O.SILU: 0.7310585786300049,
                                            O.GELU: 0.8413447460685429}[kind])
    for err, size in zip(O.act_error(g, kind, 2.0 ** -24), (value, slope)):
        assert (err >= 2.0 ** -24 * np.abs(size)).all() and (err < 1e-4 * (1 + np.abs(g))).all()


def test_int8_rows():
    x = np.array([[1.0, -2.0, 0.5], [0, 0, 0], [np.inf, 1, 2], [np.nan, 0, 0],
                  [2.0 ** -130, 2.0 ** -131, 0], [127, 63.5, -0.5]], np.float32)
    q, s = O.int8_quantize(x)
    assert list(q[0]) == [64, -127, 32] and s[0] == np.float32(2) / np.float32(127)
    assert not q[1].any() and s[1] == 0
    assert not q[2].any() and np.isnan(s[2]) and not q[3].any() and np.isnan(s[3])
    assert list(q[4]) == [127, 64, 0]
    assert list(q[5]) == [127, 64, 0]                # halves to the even code
    rng = np.random.default_rng(2)
    x = rng.normal(size=(20, 300)).astype(np.float32)
    q, s = O.int8_quantize(x)
    assert (np.abs(q).max(1) == 127).all()
    assert (np.abs(q * s[:, None].astype(np.float64) - x) <= 0.5001 * s[:, None]).all()
    p = O.int8_product(q, s, q, s)
    want = (q * s[:, None].astype(np.float64)) @ (q * s[:, None].astype(np.float64)).T
    assert (np.abs(p - want) <= 4 * 2.0 ** -24 * np.abs(want) + 1e-9).all()
