"""The MoE block's layers where a backward pass is itself recorded."""
import pytest
import torch

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
