"""The global gradient norm and clipping against 64 bits.

Tolerances (u = 2^-24): squares and sums are FP64, so the norm is rounded once
to FP32 (u) and the coefficient takes that norm and is rounded once more; a
scaled element adds the product's rounding: 4 u, and for a bf16 output half a
step, 2^-8."""
import math

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


def tensors(sizes, seed, kinds=(torch.bfloat16, torch.float32), std=1e-2, start=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    out = []
    for i, s in enumerate(sizes):
        n = math.prod(s) if isinstance(s, tuple) else s
        flat = torch.empty((n + start,), device=DEV).normal_(0.0, std, generator=g)
        out.append(flat.to(kinds[i % len(kinds)])[start:].view(s))
    return out


def check(grads, ratio, out_kinds=None, eps=1e-6):
    want = [f64(t) for t in grads]
    norm = O.clip(want, 1.0, eps)[0]
    max_norm = ratio * norm
    _, coef = O.clip(want, max_norm, eps)
    assert abs(float(B.ufp4_grad_norm(grads)) - norm) <= 2 * U * norm
    outs = None
    if out_kinds is not None:
        outs = [torch.empty_like(t, dtype=out_kinds[i % len(out_kinds)])
                for i, t in enumerate(grads)]
    got = B.ufp4_clip_grads(grads, max_norm, out=outs, eps=eps)
    assert got.dtype == torch.float32 and got.dim() == 0
    assert abs(float(got) - norm) <= 2 * U * norm
    for i, t in enumerate(outs if outs is not None else grads):
        e = want[i] * coef
        half = 2.0 ** -8 if t.dtype == torch.bfloat16 else U
        assert (np.abs(f64(t) - e) <= (half + 4 * U) * np.abs(e) + 1e-37).all(), i
    if outs is not None:
        for t, w in zip(grads, want):
            assert np.array_equal(f64(t), w)          # the inputs are kept


@pytest.mark.parametrize("ratio", [0.3, 0.999, 1.5])
@pytest.mark.parametrize("start", [0, 1])
def test_in_place_and_out(ratio, start):
    sizes = [1, 7, (3, 5), 64, (17, 1001), 16384, 16385, (130, 513), 0, 100003]
    check(tensors(sizes, 1, start=start), ratio)
    check(tensors(sizes, 2, start=start), ratio, out_kinds=(torch.float32, torch.float32,
                                                            torch.bfloat16))


@pytest.mark.parametrize("n", [1, 127, 128, 129, 400])
def test_many_tensors(n):
    check(tensors([(i * 37) % 300 + 1 for i in range(n)], n), 0.5)


def test_more_partial_sums_than_the_workspace():
    """Several launches with full grids: partial sums are folded between."""
    g = tensors([70000] * 600, 5, kinds=(torch.bfloat16,))
    check(g, 0.5)


def test_one_large_tensor_and_repeats():
    t = tensors([(1 << 26) + 5], 3, kinds=(torch.bfloat16,))
    a = B.ufp4_grad_norm(t)
    want = float(t[0].double().square().sum().sqrt())
    assert abs(float(a) - want) <= 2 * U * want
    for _ in range(3):
        assert torch.equal(a, B.ufp4_grad_norm(t))


def test_storage_orders():
    base = tensors([(40, 30, 20), (64, 48)], 4)
    check([base[0].permute(2, 0, 1), base[1].t()], 0.5)
    with pytest.raises(ValueError):
        B.ufp4_grad_norm([base[0][:, ::2]])
    with pytest.raises(ValueError):
        B.ufp4_clip_grads([base[1].t()], 1.0, out=[torch.empty((48, 64), device=DEV)])


def test_extreme_values():
    """Squares beyond FP32's range, in both directions."""
    for v in (1e30, 1e-30):
        g = [torch.full((1000,), v, device=DEV), torch.full((77,), v, device=DEV).bfloat16()]
        check(g, 0.5, eps=0.0)


def test_zero_gradients_and_no_elements():
    g = [torch.zeros(100, device=DEV), torch.zeros(0, device=DEV)]
    assert float(B.ufp4_clip_grads(g, 1.0)) == 0.0 and not g[0].any()
    assert float(B.ufp4_grad_norm([torch.zeros(0, device=DEV)])) == 0.0


def test_nonfinite_gradients():
    g = tensors([1000, 50], 6)
    g[1][3] = float("nan")
    assert math.isnan(float(B.ufp4_clip_grads(g, 1.0)))
    assert all(t.isnan().all() for t in g)
    g = tensors([1000, 50], 6)
    g[1][3] = float("inf")
    assert math.isinf(float(B.ufp4_clip_grads(g, 1.0)))
    assert not g[0].any() and g[1][3].isnan() and not g[1][:3].any()


def test_unclipped_in_place_keeps_every_bit():
    g = tensors([1000, 50], 8)
    before = [t.clone() for t in g]
    B.ufp4_clip_grads(g, 1e9)
    assert all(torch.equal(a, b) for a, b in zip(before, g))


def test_refusals():
    g = tensors([8, 8], 1)
    with pytest.raises(ValueError):
        B.ufp4_clip_grads(g, 1.0, out=g[:1])
    with pytest.raises(ValueError):
        B.ufp4_clip_grads(g, 1.0, out=[g[0], g[1][:4]])
    with pytest.raises(TypeError):
        B.ufp4_clip_grads(g, 1.0, out=[g[0].half(), g[1]])
    with pytest.raises(ValueError):
        B.ufp4_grad_norm([g[0], g[1].cpu()])
    with pytest.raises(Exception):
        B.ufp4_clip_grads(g, -1.0)
    with pytest.raises(Exception):
        B.ufp4_clip_grads([g[0]], 1.0, out=[g[0].view(torch.float32)]
                          if g[0].dtype == torch.float32 else [g[0].float()[:4]])
