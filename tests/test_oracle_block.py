"""The block operators' oracle against differences of its own forward pass,
closed forms and invariants."""
import numpy as np
import pytest

from oracle import block_oracle as O


def differences(f, x, step=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        g[i] = (f(a) - f(b)) / (2 * step)
    return g


def test_rmsnorm_gradient_against_differences():
    rng = np.random.default_rng(0)
    h, w = rng.normal(size=(3, 7)), 1 + 0.2 * rng.normal(size=7)
    dy, dh = rng.normal(size=(3, 7)), rng.normal(size=(3, 7))
    dx, dw, _, _ = O.rmsnorm_bwd(dy, h, w, 1e-3, dh)
    f = lambda h_, w_: (O.rmsnorm(h_, w_, 1e-3)[0] * dy).sum() + (h_ * dh).sum()
    assert np.allclose(dx, differences(lambda v: f(v, w), h), atol=1e-8)
    assert np.allclose(dw, differences(lambda v: f(h, v), w), atol=1e-8)


@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(renorm):
    rng = np.random.default_rng(1)
    x, k = rng.normal(size=(5, 6)), 3
    valid = np.array([1, 1, 0, 1, 1], bool)
    dg, dl = rng.normal(size=(5, k)), np.array([0.7, 0.3])

    def f(v):
        r = O.route(v, k, valid, renorm)
        return (r["gates"] * dg).sum() + (r["losses"] * dl).sum()

    d, _ = O.route_bwd(O.route(x, k, valid, renorm), k, dg, dl, renorm)
    assert np.allclose(d, differences(f, x), atol=1e-8)


def test_route_invariants():
    rng = np.random.default_rng(2)
    x = rng.integers(-3, 4, size=(40, 9)).astype(float)       # many ties
    x[7] = -np.inf
    x[8, 2:] = -np.inf
    valid = rng.random(40) < 0.8
    r = O.route(x, 4, valid)
    rows = np.where(r["slots"] < 0, ~r["slots"], r["slots"]).reshape(-1)
    assert sorted(rows) == list(range(160))                    # a permutation
    assert r["counts"].sum() == (r["experts"] >= 0).sum() and r["offsets"][-1] == 160
    for e in range(9):                                         # by expert, then by token
        mine = r["slots"][r["experts"] == e]
        assert list(mine) == list(range(r["offsets"][e], r["offsets"][e] + r["counts"][e]))
    assert (np.diff(np.take_along_axis(x, np.maximum(r["experts"], 0), 1)[valid & r["live"]],
                    axis=1)[:, :1] <= 0).all()
    # uniform probabilities and counts: the balance loss is 1
    u = O.route(np.zeros((8, 4)), 4)
    assert np.isclose(u["losses"][0], 1.0) and np.isclose(u["losses"][1], np.log(4.0) ** 2)


def test_exchange_is_linear_and_transposed():
    """<dispatch(x), v> = <x, dispatch_bwd(v)>, and combine's gradient."""
    rng = np.random.default_rng(3)
    slots = O.route(rng.normal(size=(6, 5)), 2, rng.random(6) < 0.7)["slots"]
    x, v = rng.normal(size=(6, 3)), rng.normal(size=(12, 3))
    assert np.isclose((O.dispatch(x, slots) * v).sum(), (x * O.dispatch_bwd(v, slots)[0]).sum())
    g, dy = rng.random((6, 2)), rng.normal(size=(6, 3))
    dys, dg, _ = O.combine_bwd(dy, v, slots, g)
    f = lambda v_, g_: (O.combine(v_, slots, g_)[0] * dy).sum()
    assert np.allclose(dys, differences(lambda a: f(a, g), v), atol=1e-8)
    assert np.allclose(dg, differences(lambda a: f(v, a), g), atol=1e-8)


def test_round_bf16_ties_to_even():
    x = np.array([1.0 + 2 ** -8, 1.0 + 3 * 2 ** -8, 1.0 + 2 ** -8 + 2 ** -20, -3.0, 0.0], np.float32)
    assert list(O.round_bf16(x)) == [1.0, 1.0 + 2 ** -6, 1.0 + 2 ** -7, -3.0, 0.0]
