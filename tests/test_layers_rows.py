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


def test_gradients_that_arrive_broadcast(monkeypatch):
    """Of a sum over the rows, dY is one row with stride 0, which the library
    does not take as rows: it is written out."""
    seen = []

    def quantize(t, *a, **kw):
        seen.append(t)
        return t, t.t()

    monkeypatch.setattr(Y.U, "ufp4_rht_quantize_dual", quantize)
    for layer, more in ((Y.UFP4Linear(8, 4), ()),
                        (Y.UFP4ExpertLinear(1, 8, 4), (torch.tensor([0, 5]),))):
        for grad in (torch.ones((), dtype=torch.bfloat16).expand(5, 4),
                     torch.arange(4).to(torch.bfloat16).expand(5, 4),
                     torch.arange(5).to(torch.bfloat16)[:, None].expand(5, 4)):
            x = torch.ones((5, 8), dtype=torch.bfloat16, requires_grad=True)
            layer(x, *more).backward(grad)
            dy = seen[-1]
            assert dy.stride(1) == 1 and dy.stride(0) >= 4 and torch.equal(dy, grad)
    wide = torch.ones((5, 20), dtype=torch.bfloat16)[:, 3:11]      # rows of any stride stay
    Y.UFP4Linear(8, 4)(wide)
    assert seen[-2].data_ptr() == wide.data_ptr()
