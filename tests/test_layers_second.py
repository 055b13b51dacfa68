"""The linear and expert layers without a GPU, where a backward pass is itself
recorded: the library's calls stand in as plain products."""
import pytest
import torch

from uniform_grid_fp4_amd import layers as Y


@pytest.fixture(autouse=True)
def plain(monkeypatch):
    monkeypatch.setattr(Y.U, "ufp4_rht_quantize_dual", lambda t, *a, **kw: (t, t.t()))
    monkeypatch.setattr(Y.U, "ufp4_gemm_out", lambda kind, a, b, dtype: a @ b.t())
    monkeypatch.setattr(Y.U, "ufp4_grouped_gemm_out", lambda kind, off, a, b, dtype: a @ b.t())


def bf(*shape):
    return (torch.arange(torch.Size(shape).numel(), dtype=torch.float32).reshape(shape) % 5
            - 2.0).to(torch.bfloat16)


@pytest.mark.parametrize("make", [lambda: (Y.UFP4Linear(8, 4), ()),
                                  lambda: (Y.UFP4ExpertLinear(1, 8, 4),
                                           (torch.tensor([0, 3]),))])
def test_second_derivatives_are_refused(make):
    layer, more = make()
    for loss in (torch.sum, lambda y: y.square().sum()):
        x = bf(3, 8).requires_grad_()
        want = torch.autograd.grad(loss(layer(x, *more)), [x, layer.weight])
        got = torch.autograd.grad(loss(layer(x, *more)), [x, layer.weight], create_graph=True)
        for a, b in zip(want, got):
            assert torch.equal(a, b)
            with pytest.raises(RuntimeError, match="second derivative"):
                (b.sum() + x.sum()).backward(retain_graph=True)
    # X alone is differentiated and the gradient of a sum is a constant of X
    layer.weight.requires_grad_(False)
    x = bf(3, 8).requires_grad_()
    g, = torch.autograd.grad(layer(x, *more).sum(), x, create_graph=True)
    (g.sum() + x.sum()).backward()
    assert torch.equal(x.grad, torch.ones_like(x))
