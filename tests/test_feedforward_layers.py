"""The feed-forward layers without a GPU: what they do around the library's
calls, which stand in as plain products here."""
import pytest
import torch

from uniform_grid_fp4_amd import feedforward as W
from uniform_grid_fp4_amd import layers as Y
from uniform_grid_fp4_amd import moe as M


@pytest.fixture
def plain(monkeypatch):
    def gated(xq, wq, act, keep, offsets):
        gu = xq @ wq.t()
        f = gu.shape[1] // 2
        return W.F.GatedOut(gu[:, :f] * gu[:, f:], gu.clone() if keep else None)

    def gated_bwd(dy, gu, act, out):
        f = dy.shape[1]
        return out.copy_(torch.cat([dy * gu[:, f:], dy * gu[:, :f]], 1))

    monkeypatch.setattr(Y.U, "ufp4_rht_quantize_dual", lambda t, *a, **kw: (t, t.t()))
    monkeypatch.setattr(Y.U, "ufp4_gemm_out", lambda kind, a, b, dtype: a @ b.t())
    monkeypatch.setattr(Y.U, "ufp4_grouped_gemm_out", lambda kind, off, a, b, dtype: a @ b.t())
    monkeypatch.setattr(W.F, "ufp4_gated_gemm", gated)
    monkeypatch.setattr(W.F, "ufp4_gated_bwd", gated_bwd)
    monkeypatch.setattr(W.F, "ufp4_layernorm", lambda x, w, b, res, eps: W.F.LayerNormOut(
        x * w + (0 if b is None else b), x if res is None else x + res, x.sum(1), x.sum(1)))
    monkeypatch.setattr(W.F, "ufp4_layernorm_bwd", lambda dy, h, w, m, r, dh, bias: (
        dy * w + (0 if dh is None else dh), (dy * h).sum(0), dy.sum(0) if bias else None))
    monkeypatch.setattr(W.F, "ufp4_dropout", lambda x, p, seed, offset, residual=None: (
        x * (0.0 if p else 1.0) + (0 if residual is None else residual)))


def bf(*shape):
    return (torch.arange(torch.Size(shape).numel(), dtype=torch.float32).reshape(shape) % 5
            - 2.0).to(torch.bfloat16)


MAKES = [lambda: (W.UFP4GatedLinear(8, 4), ()),
         lambda: (W.UFP4GatedExpertLinear(1, 8, 4), (torch.tensor([0, 3]),))]


@pytest.mark.parametrize("make", MAKES)
def test_gated_gradients_are_those_of_the_product(plain, make):
    layer, more = make()
    x = bf(3, 8).requires_grad_()
    y = layer(x, *more)
    dy = bf(3, 4) + 1
    dx, dw = torch.autograd.grad(y, [x, layer.weight], dy)
    x2, w2 = x.detach().clone().requires_grad_(), layer.weight.detach().clone().requires_grad_()
    gu = x2 @ w2.t()
    want = torch.autograd.grad(gu[:, :4] * gu[:, 4:], [x2, w2], dy)
    for a, b in zip((dx, dw), want):
        assert a.shape == b.shape and torch.allclose(a.float(), b.float(), rtol=0.05, atol=0.05)


@pytest.mark.parametrize("make", MAKES)
def test_gated_layers_keep_what_a_backward_pass_needs_and_no_more(plain, make):
    layer, more = make()
    kept = []
    call = W.F.ufp4_gated_gemm
    W.F.ufp4_gated_gemm = lambda *a, keep, **kw: kept.append(keep) or call(*a, keep=keep, **kw)
    try:
        with torch.no_grad():
            layer(bf(3, 8), *more)
        layer(bf(3, 8), *more)
        layer.weight.requires_grad_(False)
        layer(bf(3, 8), *more)
        y = layer(bf(3, 8).requires_grad_(), *more)
    finally:
        W.F.ufp4_gated_gemm = call
    assert kept == [False, True, False, True]
    y.sum().backward(retain_graph=True)
    with pytest.raises(RuntimeError, match="has run"):
        y.sum().backward()


@pytest.mark.parametrize("make", MAKES)
def test_gated_second_derivatives_are_refused(plain, make):
    layer, more = make()
    x = bf(3, 8).requires_grad_()
    grads = torch.autograd.grad(layer(x, *more).sum(), [x, layer.weight], create_graph=True)
    for g in grads:
        with pytest.raises(RuntimeError, match="second derivative"):
            (g.sum() + x.sum()).backward(retain_graph=True)


@pytest.mark.parametrize("make", MAKES)
def test_batches_without_rows(plain, make):
    layer, more = make()
    x = torch.empty((0, 8), dtype=torch.bfloat16, requires_grad=True)
    if more:
        more = (torch.tensor([0, 0]),)
    y = layer(x, *more)
    assert y.shape == (0, 4)
    y.sum().backward()
    assert x.grad.shape == (0, 8) and not layer.weight.grad.any()


def test_layer_arguments():
    with pytest.raises(ValueError, match="act"):
        W.UFP4GatedLinear(8, 4, act="relu")
    with pytest.raises(ValueError, match="probability"):
        W.Dropout(1.5)
    with pytest.raises(TypeError):
        W.UFP4GatedLinear(8, 4)(torch.zeros(3, 8))
    with pytest.raises(ValueError):
        W.Int8Linear(torch.zeros(9, 4), n_experts=2)
    with pytest.raises(ValueError):
        W.Int8Linear(torch.zeros(9, 4), act="silu")
    with pytest.raises(TypeError, match="gated"):
        W.Int8MoEBlock(M.UFP4MoEBlock(8, 4, 2, 1))
    assert isinstance(M.UFP4MoEBlock(8, 4, 2, 1, gated="gelu").up, W.UFP4GatedExpertLinear)
    assert isinstance(M.UFP4MoEBlock(8, 4, 2, 1).up, Y.UFP4ExpertLinear)


def test_a_residual_of_another_shape_is_refused():
    """As rows they would fit, each meeting another's."""
    x, r = torch.zeros(2, 3, 8), torch.zeros(3, 2, 8)
    for call in (W.LayerNorm(8), W.Dropout(0.5), W.Dropout(0.0)):
        with pytest.raises(ValueError, match="shape"):
            call(x, r)


def test_layer_norm_gradients(plain):
    norm = W.LayerNorm(4, dtype=torch.float32)
    x, r = torch.randn(2, 3, 4, requires_grad=True), torch.randn(2, 3, 4, requires_grad=True)
    y, h = norm(x, r)
    assert y.shape == h.shape == x.shape
    (y.sum() + 2 * h.sum()).backward()
    assert torch.equal(x.grad, r.grad) and torch.equal(x.grad, torch.full_like(x, 3.0))
    assert torch.equal(norm.bias.grad, torch.full((4,), 6.0))
    x.grad = None
    norm(x, r)[1].sum().backward()
    assert torch.equal(x.grad, torch.ones_like(x))
    bare = W.LayerNorm(4, bias=False, dtype=torch.float32)
    bare(x).sum().backward()
    assert bare.bias is None and bare.weight.grad is not None
    g, = torch.autograd.grad(norm(x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        (g.sum() + x.sum()).backward()


def test_dropout_layer(plain, monkeypatch):
    seen = []
    call = W.F.ufp4_dropout
    monkeypatch.setattr(W.F, "ufp4_dropout", lambda x, p, seed, offset, residual=None: seen.append(
        (p, seed, offset)) or call(x, p, seed, offset, residual))
    drop = W.Dropout(0.25, seed=5)
    x, r = torch.randn(2, 3, 4, requires_grad=True), torch.randn(2, 3, 4, requires_grad=True)
    drop(x, r).sum().backward()
    drop(x).sum().backward()
    # forward and backward of a call name the same mask, the next call another
    assert seen == [(0.25, 5, 1), (0.25, 5, 1), (0.25, 5, 2), (0.25, 5, 2)]
    assert torch.equal(r.grad, torch.ones_like(r)) and not x.grad.any()
    drop.eval()
    assert drop(x) is x
    assert torch.equal(drop(x, r), x + r) and seen[-1][0] == 0.0 and drop.calls == 2
    step = torch.tensor([7])
    drop = W.Dropout(0.5, offset=step)
    y = drop(x)
    assert seen[-1][2] is step
    y.sum().backward()
    # a mask whose offset has moved on cannot be drawn again
    y = drop(x)
    step += 1
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()
