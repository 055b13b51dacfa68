"""The linear and expert layers without rows, without a GPU: the library's calls
stand in as plain products that refuse an empty tensor, as the library does."""
import pytest
import torch

from uniform_grid_fp4_amd import layers as Y


@pytest.fixture(autouse=True)
def plain(monkeypatch):
    def quantize(t, *a, **kw):
        if t.shape[0] == 0:
            raise Y.U.UFP4Error(-2, "ufp4_rht_quantize_dual")
        return t, t.t()

    monkeypatch.setattr(Y.U, "ufp4_rht_quantize_dual", quantize)
    monkeypatch.setattr(Y.U, "ufp4_gemm_out", lambda kind, a, b, dtype: a @ b.t())
    monkeypatch.setattr(Y.U, "ufp4_grouped_gemm_out", lambda kind, off, a, b, dtype: a @ b.t())


@pytest.mark.parametrize("lead", [(0,), (2, 0)])
def test_no_rows(lead):
    x = torch.zeros((*lead, 8), dtype=torch.bfloat16, requires_grad=True)
    for layer, more in ((Y.UFP4Linear(8, 4), ()),
                        (Y.UFP4ExpertLinear(3, 8, 4), (torch.zeros(4, dtype=torch.int64),))):
        seed = layer.sr_seed
        y = layer(x, *more)
        assert y.shape[-1] == 4 and y.numel() == 0 and y.dtype == torch.bfloat16
        assert layer.sr_seed == seed + 1
        x.grad = None
        y.float().sum().backward()
        assert x.grad.shape == x.shape
        assert layer.weight.grad.shape == layer.weight.shape and not layer.weight.grad.any()
    with pytest.raises(TypeError):
        Y.UFP4Linear(8, 4)(torch.zeros((0, 8)))
