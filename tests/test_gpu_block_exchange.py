"""Dispatch, combine and their backward passes against the 64-bit oracle.

Tolerances (u = 2^-24): a sum of k choices is within (k + 4) u of its terms'
magnitudes, a row's dot product within (n / 64 + 32) u, and a bf16 result adds
half a step, 2^-8.  Dispatch copies."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as O
from uniform_grid_fp4_amd import block as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def close(got, want, size, c, what):
    half = HALF[got.dtype]
    lim = c * size + half * (np.abs(want) + c * size) + 1e-37
    err = np.abs(f64(got) - want)
    assert (err <= lim).all(), f"{what}: worst ratio {(err / lim).max():.3g}"


def make(t, cols, k, dtype, seed, padded=0.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n = lambda r, std: torch.empty((r, cols), device=DEV).normal_(0.0, std, generator=g).to(dtype)
    off = torch.rand((t, k), device=DEV, generator=g) < padded
    key = torch.rand((t, k), device=DEV, generator=g) + off
    rows = key.reshape(-1).argsort().argsort().reshape(t, k).to(torch.int32)
    slots = torch.where(off, ~rows, rows)
    gates = torch.rand((t, k), device=DEV, generator=g) * ~off
    return slots, gates, n(t, 1.0), n(t * k, 1.0), n(t, 1.0), n(t, 1.0), n(t * k, 1.0)


def check(t, cols, k, dtype, padded=0.0, seed=0):
    print(f"[exchange] {t} x {cols}, k {k}, {dtype}, padded {padded}", flush=True)
    slots, gates, x, ys, res, dy, dxs = make(t, cols, k, dtype, seed + t + cols, padded)
    s, g = slots.cpu().numpy(), gates.cpu().numpy()
    assert np.array_equal(f64(B.ufp4_moe_dispatch(x, slots)), O.dispatch(f64(x), s))
    # rows without a choice are not read: NaN there changes nothing
    lost = np.unique(np.where(s < 0, ~s, -1))
    for r in lost[lost >= 0]:
        ys[int(r)] = float("nan")
        dxs[int(r)] = float("nan")
    yc = np.nan_to_num(f64(ys), nan=0.0)
    close(B.ufp4_moe_dispatch_bwd(dxs, slots), *O.dispatch_bwd(np.nan_to_num(f64(dxs)), s),
          (k + 4) * U, "dx")
    for r in (None, res):
        close(B.ufp4_moe_combine(ys, slots, gates, r),
              *O.combine(yc, s, g, None if r is None else f64(r)), (k + 4) * U, "y")
    dys, dg = B.ufp4_moe_combine_bwd(dy, ys, slots, gates)
    ed, eg, size = O.combine_bwd(f64(dy), yc, s, g)
    close(dys, ed, np.abs(ed), U, "dys")
    assert (np.abs(f64(dg) - eg) <= (cols / 64 + 32) * U * size + 1e-37).all()
    return slots, gates, x, ys, res, dy, dxs


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,cols,k", [(1, 1, 1), (1, 2048, 8), (3, 7, 2), (16, 6144, 8),
                                      (65, 100, 3), (33, 511, 5), (20, 2049, 6), (9, 8192, 7),
                                      (40, 64, 16), (12, 4097, 12), (500, 264, 4)])
def test_exchange(t, cols, k, dtype):
    check(t, cols, k, dtype)
    check(t, cols, k, dtype, padded=0.3, seed=7)


def test_every_choice_missing():
    slots, gates, x, ys, res, dy, dxs = check(10, 96, 3, torch.bfloat16, padded=1.0)
    assert not B.ufp4_moe_dispatch(x, slots).any()
    assert torch.equal(B.ufp4_moe_combine(ys, slots, gates, res), res)


def test_slots_outside_the_array_have_no_row():
    """Such choices are left out, and nothing is touched outside."""
    slots, gates, x, ys, res, dy, dxs = make(8, 64, 2, torch.bfloat16, 4)
    bad = slots.clone()
    bad[3, 1], bad[5, 0], bad[6, 1] = 16, 2 ** 31 - 1, -(2 ** 31)
    ok = bad.clone()
    ok[3, 1] = ok[5, 0] = ok[6, 1] = ~0
    assert torch.equal(B.ufp4_moe_dispatch_bwd(dxs, bad), B.ufp4_moe_dispatch_bwd(dxs, ok))
    assert torch.equal(B.ufp4_moe_combine(ys, bad, gates), B.ufp4_moe_combine(ys, ok, gates))
    a = B.ufp4_moe_combine_bwd(dy, ys, bad, gates)[1]
    assert torch.equal(a, B.ufp4_moe_combine_bwd(dy, ys, ok, gates)[1])
    xs = B.ufp4_moe_dispatch(x, bad)
    for t in range(8):
        for j in range(2):
            if 0 <= int(bad[t, j]) < 16:
                assert torch.equal(xs[int(bad[t, j])], x[t])


def test_strided_rows():
    slots, gates, x, ys, res, dy, dxs = make(12, 100, 4, torch.bfloat16, 6)
    wide = torch.full((3, 12, 111), float("nan"), dtype=torch.bfloat16, device=DEV)
    for i, v in enumerate((x, res, dy)):
        wide[i, :, 5:105] = v
    vx, vr, vd = (wide[i, :, 5:105] for i in range(3))
    assert torch.equal(B.ufp4_moe_dispatch(x, slots), B.ufp4_moe_dispatch(vx, slots))
    assert torch.equal(B.ufp4_moe_combine(ys, slots, gates, res),
                       B.ufp4_moe_combine(ys, slots, gates, vr))
    for u, v in zip(B.ufp4_moe_combine_bwd(dy, ys, slots, gates),
                    B.ufp4_moe_combine_bwd(vd, ys, slots, gates)):
        assert torch.equal(u, v)


def test_zero_tokens():
    slots = torch.zeros((0, 4), dtype=torch.int32, device=DEV)
    gates = torch.zeros((0, 4), device=DEV)
    e = torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV)
    assert B.ufp4_moe_dispatch(e, slots).shape == (0, 64)
    assert B.ufp4_moe_dispatch_bwd(e, slots).shape == (0, 64)
    assert B.ufp4_moe_combine(e, slots, gates, e).shape == (0, 64)
    assert B.ufp4_moe_combine_bwd(e, e, slots, gates)[1].shape == (0, 4)


def test_offsets_past_32_bits():
    """An array whose element offsets pass 2^32 (8.6 GB in bf16): its first,
    last and some other rows."""
    t, cols, k = 70000, 8192, 8
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    rows = torch.randperm(t * k, device=DEV, generator=g).reshape(t, k).to(torch.int32)
    x = torch.randint(-8, 9, (t, cols), device=DEV, generator=g).to(torch.bfloat16)
    xs = B.ufp4_moe_dispatch(x, rows)
    dx = B.ufp4_moe_dispatch_bwd(xs, rows)
    assert torch.equal(dx, x * k)                     # exact: small whole numbers
    for i in (0, 1, t * k - 2, t * k - 1, 524288, 524289):
        at = (rows == i).nonzero()[0]
        assert torch.equal(xs[i], x[at[0]])


def test_refusals():
    slots, gates, x, ys, res, dy, _ = make(8, 64, 2, torch.bfloat16, 1)
    with pytest.raises(ValueError):
        B.ufp4_moe_dispatch(x[:7], slots)
    with pytest.raises(TypeError):
        B.ufp4_moe_dispatch(x, slots.long())
    with pytest.raises(ValueError):
        B.ufp4_moe_dispatch(x, slots.cpu())
    with pytest.raises(ValueError):
        B.ufp4_moe_combine(ys[:-1], slots, gates)
    with pytest.raises(TypeError):
        B.ufp4_moe_combine(ys, slots, gates, res.float())
    with pytest.raises(ValueError):
        B.ufp4_moe_combine(ys, slots, gates[:, :1])
    with pytest.raises(ValueError):
        B.ufp4_moe_combine_bwd(dy[:4], ys, slots, gates)
    with pytest.raises(ValueError):
        B.ufp4_moe_dispatch(x, torch.zeros((8, 17), dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        B.ufp4_moe_combine(ys.repeat(1, 2)[:, ::2], slots, gates)
