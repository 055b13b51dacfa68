"""Serving layers of a model that was cast as a whole answer as before."""
import pytest
import torch

from uniform_grid_fp4_amd import feedforward as W
from uniform_grid_fp4_amd import moe as M

pytestmark = pytest.mark.gpu


def test_cast_models_serve():
    torch.manual_seed(0)
    x = torch.randn(9, 128, device="cuda").to(torch.bfloat16)
    served = W.Int8FeedForward(W.UFP4FeedForward(128, 192, device="cuda"))
    block = W.Int8MoEBlock(M.UFP4MoEBlock(128, 96, 4, 2, device="cuda", gated="silu"))
    want = served(x), block(x).y
    assert torch.equal(served.to(torch.bfloat16)(x), want[0])
    assert torch.equal(block.up.to(torch.bfloat16).scale, block.up.scale)
    block.down.half()
    assert torch.equal(block(x).y, want[1])
