"""The MoE block without a token."""
import pytest
import torch

from uniform_grid_fp4_amd import moe as M

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("lead", [(0,), (3, 0)])
def test_block_without_tokens(lead):
    """As the operators it consists of: nothing comes out, and every gradient is
    zero."""
    block = M.UFP4MoEBlock(64, 32, 4, 2, device=DEV)
    x, r = (torch.zeros((*lead, 64), dtype=torch.bfloat16, device=DEV, requires_grad=True)
            for _ in range(2))
    valid = torch.zeros(lead, dtype=torch.bool, device=DEV)
    for residual in (None, r):
        out = block(x, residual, valid)
        assert out.y.shape == x.shape and out.residual.shape == x.shape
        assert not out.counts.any() and not out.losses.any()
        block.zero_grad()
        (out.y.float().sum() + out.losses.sum()).backward()
        assert x.grad.shape == x.shape
        for name, p in block.named_parameters():
            assert p.grad is not None and not p.grad.any(), name
    assert float(M.clip_grad_norm_(block.parameters(), 1.0)) == 0.0
