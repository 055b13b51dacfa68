"""The MoE router, forward and backward, against the 64-bit oracle.

Whole numbers are equal.  Floating tolerances (u = 2^-24): with d the largest
distance between a row's logits and its lse, an argument of exp is rounded by
up to d u and so is its value relative to itself; a row sum over E experts is a
chain of E / 16 additions and 8 more; 32 u cover the functions and products.
So values are within c = (2 d + E / 16 + 40) u of their terms' magnitudes; a
sum over tokens adds a chain of at most 16 u.  bf16 adds half a step, 2^-8."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as O
from uniform_grid_fp4_amd import block as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def logits_of(t, e, dtype, seed, std=1.5):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.empty((t, e), device=DEV).normal_(0.0, std, generator=g)
            + torch.empty((e,), device=DEV).normal_(0.0, 0.7, generator=g)).to(dtype)


def within(got, want, lim, what):
    g = f64(got)
    assert np.array_equal(np.isfinite(g), np.isfinite(want)), what
    fine = np.isfinite(want)
    err, lim = np.abs(g[fine] - want[fine]), (lim + np.zeros_like(want))[fine]
    assert (err <= lim).all(), f"{what}: worst ratio {(err / np.maximum(lim, 1e-300)).max():.3g}"
    assert np.array_equal(g[~fine], want[~fine]), what


def check(x, k, valid=None, renorm=True, grad=True, seed=0):
    t, e = x.shape
    print(f"[route] {t} x {e}, k {k}, {x.dtype}, renorm {renorm}", flush=True)
    r = B.ufp4_moe_route(x, k, valid=valid, renorm=renorm)
    o = O.route(f64(x), k, None if valid is None else valid.cpu().numpy(), renorm)
    for name in ("experts", "slots", "counts", "offsets"):
        assert np.array_equal(getattr(r, name).cpu().numpy(), o[name]), name
    assert int(r.n_tokens) == o["n_tokens"]
    live, xs = o["live"], f64(x)
    d = 1.0
    if live.any():
        lse = o["lse"][live][:, None]
        # a distance over 90 leaves nothing in FP32
        d = min(90.0, float(np.abs(np.where(np.isfinite(xs[live]), xs[live], lse) - lse).max()))
    c = (2 * d + e / 16 + 40) * U
    within(r.gates, o["gates"], c * o["gates"] + 1e-36, "gates")
    fin = np.where(live, np.abs(o["lse"]), 0.0)
    within(r.lse, o["lse"], c + 4 * U * np.where(live, fin, 1.0), "lse")
    n = max(1, o["n_tokens"])
    zerr = (2 * fin * (c + 4 * U * fin) + (c + 4 * U * fin) ** 2).sum() / n
    with np.errstate(over="ignore"):                  # a z loss beyond FP32 is infinite
        losses = o["losses"].astype(np.float32).astype(np.float64)
    within(r.losses, losses, np.array([(c + 16 * U) * losses[0] + 1e-36,
                                       zerr + 4 * U * o["losses"][1]]), "losses")
    if grad:
        g = torch.Generator(device=DEV)
        g.manual_seed(seed + 5)
        dg = torch.empty((t, k), device=DEV).normal_(0.0, 1e-2, generator=g)
        dl = torch.tensor([0.3, 0.02], device=DEV)
        half = 2.0 ** -8 if x.dtype == torch.bfloat16 else U
        for pair in ((dg, dl), (dg, None), (None, dl)):
            got = B.ufp4_moe_route_bwd(x, r, *pair)
            want, size = O.route_bwd(o, k, f64(dg) * (pair[0] is not None),
                                     f64(dl) * (pair[1] is not None), renorm)
            assert got.dtype == x.dtype
            within(got, want, 2 * c * size + half * (np.abs(want) + 2 * c * size) + 1e-36,
                   "d_logits")
    return r


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 64, 6), (2, 8, 8), (63, 5, 2), (64, 16, 4),
                                   (65, 17, 3), (128, 64, 6), (200, 100, 7), (130, 130, 16),
                                   (77, 256, 8), (300, 250, 8), (66, 512, 10), (70, 600, 9),
                                   (100, 1024, 16), (65, 1023, 1)])
def test_router(t, e, k, dtype):
    x = logits_of(t, e, dtype, t * 1000 + e)
    for renorm in (True, False):
        check(x, k, None, renorm, seed=t)


def test_many_workgroups():
    x = logits_of(9000, 64, torch.float32, 4)
    valid = torch.rand(9000, device=DEV) < 0.8
    check(x, 6, valid, False)
    a = B.ufp4_moe_route(x, 6, valid=valid)
    for _ in range(3):                                # bit for bit, whatever ran first
        b = B.ufp4_moe_route(x, 6, valid=valid)
        for u, v in zip(a[:8], b[:8]):
            assert torch.equal(u, v)


@pytest.mark.parametrize("t", [1, 64, 500])
def test_no_token_takes_part(t):
    x = logits_of(t, 32, torch.float32, 3)
    check(x, 4, torch.zeros(t, dtype=torch.bool, device=DEV))
    check(torch.full_like(x, -float("inf")), 4)


def test_zero_tokens():
    r = B.ufp4_moe_route(torch.zeros((0, 16), device=DEV), 2)
    assert r.slots.shape == (0, 2) and not r.counts.any() and not r.offsets.any()
    assert not r.losses.any() and int(r.n_tokens) == 0
    assert B.ufp4_moe_route_bwd(torch.zeros((0, 16), device=DEV), r).shape == (0, 16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_masks_and_lowest_values(dtype):
    """Equal logits (and -0 with +0) go to the lowest expert; -inf is never
    chosen, the type's lowest finite value is; rows with fewer experts than
    choices; a wide range."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randint(-2, 3, (150, 40), device=DEV, generator=g).to(dtype)
    x[3] = 0.0
    x[3, ::2] = -0.0
    x[4] = torch.finfo(dtype).min
    x[5] = -float("inf")
    x[6] = -float("inf")
    x[6, 7] = 1.0
    x[7, 1:] = -float("inf")
    x[8, 2:] = torch.finfo(dtype).min
    x[9, 5:] = -float("inf")
    x[9, :5] = torch.finfo(dtype).min
    x[10, 3] = 80.0
    x[11] = torch.finfo(dtype).max / 4
    for renorm in (True, False):
        check(x, 6, None, renorm, grad=False)
        check(x[:64], 6, None, renorm, grad=False)
    keep = [i for i in range(150) if i != 11]
    check(x[keep], 6, None, True)


def test_nan_and_inf_rows_do_not_reach_others():
    x = logits_of(200, 48, torch.float32, 8)
    want = B.ufp4_moe_route(x, 4)
    y = x.clone()
    y[20, 3] = float("nan")
    y[30, 4] = float("inf")
    y[40] = float("nan")
    r = B.ufp4_moe_route(y, 4)
    rows = torch.where(r.slots < 0, ~r.slots, r.slots).reshape(-1)
    assert torch.equal(rows.sort().values.cpu(), torch.arange(800, dtype=torch.int32))
    assert int(r.counts.sum()) == int((r.experts >= 0).sum()) == 800 - 4
    assert not (r.experts[20] == 3).any() and (r.experts[30, 0] == 4) and (r.experts[40] < 0).all()
    assert r.gates[20].isnan().all() and r.losses.isnan().all() and r.lse[40].isnan()
    keep = [i for i in range(200) if i not in (20, 30, 40)]
    assert torch.equal(want.gates[keep], r.gates[keep])
    assert torch.equal(want.experts[keep], r.experts[keep])
    d = B.ufp4_moe_route_bwd(y, r, torch.ones((200, 4), device=DEV))
    assert d[keep].isfinite().all() and d[20].isnan().all()


def test_strided_logits():
    for dtype in (torch.float32, torch.bfloat16):
        x = logits_of(90, 64, dtype, 2)
        wide = torch.full((90, 71), float("nan"), dtype=dtype, device=DEV)
        wide[:, 3:67] = x
        a, b = B.ufp4_moe_route(x, 6), B.ufp4_moe_route(wide[:, 3:67], 6)
        for u, v in zip(a[:8], b[:8]):
            assert torch.equal(u, v)
        dg = torch.rand((90, 6), device=DEV)
        assert torch.equal(B.ufp4_moe_route_bwd(x, a, dg),
                           B.ufp4_moe_route_bwd(wide[:, 3:67], b, dg))


def test_gradient_against_differences():
    """The kernel's gradient against central differences of the oracle's
    forward pass in 64 bits (step 1e-6: truncation and cancellation below
    1e-8, FP32 results within c of terms of at most 1)."""
    x = logits_of(6, 10, torch.float32, 12)
    valid = torch.tensor([1, 1, 0, 1, 1, 1], dtype=torch.bool, device=DEV)
    dg = torch.rand((6, 3), device=DEV)
    dl = torch.tensor([0.5, 0.25], device=DEV)
    for renorm in (True, False):
        r = B.ufp4_moe_route(x, 3, valid=valid, renorm=renorm)
        got = f64(B.ufp4_moe_route_bwd(x, r, dg, dl))
        base, want = f64(x), np.zeros((6, 10))

        def f(v):
            o = O.route(v, 3, valid.cpu().numpy(), renorm)
            return (o["gates"] * f64(dg)).sum() + (o["losses"] * f64(dl)).sum()

        for i in np.ndindex(6, 10):
            up, down = base.copy(), base.copy()
            up[i] += 1e-6
            down[i] -= 1e-6
            want[i] = (f(up) - f(down)) / 2e-6
        assert np.abs(got - want).max() < 1e-5


def test_refusals():
    x = logits_of(8, 16, torch.float32, 1)
    r = B.ufp4_moe_route(x, 4)
    for k in (0, 17):
        with pytest.raises(ValueError):
            B.ufp4_moe_route(x, k)
    with pytest.raises(ValueError):
        B.ufp4_moe_route(torch.zeros((4, 40), device=DEV), 17)
    with pytest.raises(TypeError):
        B.ufp4_moe_route(x, 4, valid=torch.ones(8, device=DEV))
    with pytest.raises(ValueError):
        B.ufp4_moe_route(x, 4, valid=torch.ones(7, dtype=torch.bool, device=DEV))
    with pytest.raises(ValueError):
        B.ufp4_moe_route_bwd(x[:7], r)
    with pytest.raises(TypeError):
        B.ufp4_moe_route_bwd(x, r, r.gates.double())
    with pytest.raises(Exception):
        B.ufp4_moe_route(torch.zeros((4, 1025), device=DEV), 2)
