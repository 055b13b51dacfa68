"""The MoE block's layers without a GPU: what they do around the library's
calls."""
import pytest
import torch

from uniform_grid_fp4_amd import moe as M


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_clipping_without_gradients_gives_a_zero_where_the_parameters_are(device):
    p = torch.nn.Parameter(torch.empty(3, device=device))
    for params in (p, [p, p], iter([p])):
        norm = M.clip_grad_norm_(params, 1.0)
        assert norm.device == p.device and norm.dtype == torch.float32 and norm.dim() == 0
    assert float(M.clip_grad_norm_([], 1.0)) == 0.0          # no parameters: nowhere else to be
