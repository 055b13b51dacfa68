"""Clipping where the coefficient's quotient has no value of its own."""
import math

import pytest
import torch

from uniform_grid_fp4_amd import block as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_zero_gradients_stay_zero_whatever_the_limit():
    """A norm of zero is within any limit, also one of zero without an eps."""
    for max_norm in (0.0, 1.0):
        for eps in (0.0, 1e-6):
            g = [torch.zeros(100, device=DEV), torch.zeros(7, dtype=torch.bfloat16, device=DEV)]
            out = [torch.full_like(t, 3.0) for t in g]
            assert float(B.ufp4_clip_grads(g, max_norm, out=out, eps=eps)) == 0.0
            B.ufp4_clip_grads(g, max_norm, eps=eps)
            for t in (*g, *out):
                assert not t.any() and not t.isnan().any()


def test_no_limit_scales_nothing():
    """An infinite limit leaves finite and infinite gradients as they are; a NaN
    still gives NaN everywhere."""
    inf = float("inf")
    g = [torch.tensor([1.0, inf, -2.0], device=DEV), torch.ones(5, device=DEV)]
    want = [t.clone() for t in g]
    assert math.isinf(float(B.ufp4_clip_grads(g, inf)))
    assert all(torch.equal(a, b) for a, b in zip(g, want))
    out = [torch.empty_like(t) for t in g]
    B.ufp4_clip_grads(g, inf, out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    g[1][2] = float("nan")
    assert math.isnan(float(B.ufp4_clip_grads(g, inf)))
    assert all(t.isnan().all() for t in g)


def test_a_limit_of_zero_gives_zeros():
    g = [torch.ones(100, device=DEV)]
    assert float(B.ufp4_clip_grads(g, 0.0)) == 10.0 and not g[0].any()
