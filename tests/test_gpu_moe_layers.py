"""The MoE block's layers and autograd: a backward pass that is itself
recorded, and tensors that calls update in place."""
import pytest
import torch

from uniform_grid_fp4_amd import block as B
from uniform_grid_fp4_amd import moe as M

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_recorded_backward_passes():
    """The same first derivatives; second ones are refused, not cut short."""
    torch.manual_seed(0)
    norm, router = M.RMSNorm(64, device=DEV), M.MoERouter(64, 8, 2, device=DEV)
    params = [norm.weight, router.weight]

    def loss(x):
        y, h = norm(x, x)
        r = router(y)
        out = M.combine(M.dispatch(y, r.slots), r.slots, r.gates, h)
        return out.float().square().sum() + r.losses.sum()

    x = torch.randn((30, 64), device=DEV).to(torch.bfloat16).requires_grad_()
    want = torch.autograd.grad(loss(x), [x, *params])
    got = torch.autograd.grad(loss(x), [x, *params], create_graph=True)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    for g in got:
        with pytest.raises(RuntimeError, match="second derivative"):
            (g.float().sum() + x.float().sum()).backward(retain_graph=True)


def test_autograd_sees_what_is_updated_in_place():
    """A tensor that a backward pass has saved and a call then overwrites makes
    that backward pass raise, as after torch's own in-place operations."""
    rows, w = torch.randn((2, 30, 64), device=DEV).to(torch.bfloat16), torch.ones(64, device=DEV)
    scale = torch.ones(64, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    for which in (0, 1):
        x, res = rows.clone().unbind(0)
        saved = ((x, res)[which] * scale).sum()
        B.ufp4_rmsnorm(x, w, res, out_h=(x, res)[which])
        with pytest.raises(RuntimeError, match="modified by an inplace"):
            saved.backward()
        x, res = rows.clone().unbind(0)
        saved = (x * scale).sum() + (res * scale).sum()
        B.ufp4_rmsnorm(x, w, res)                        # into a tensor of its own
        saved.backward()
    grads = [torch.ones(100, device=DEV), torch.ones(7, device=DEV)]
    saved = sum((g * scale.float()[:1]).sum() for g in grads)
    B.ufp4_grad_norm(grads)
    B.ufp4_clip_grads(grads, 0.5, out=[torch.empty_like(g) for g in grads])
    saved.backward(retain_graph=True)
    B.ufp4_clip_grads(grads, 0.5)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        saved.backward()
