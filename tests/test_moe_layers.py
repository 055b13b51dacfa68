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


@pytest.fixture
def plain(monkeypatch):
    """The library's calls as products of what they take, enough for autograd to
    have something to record or to refuse."""
    r = lambda x, k, **kw: M.B.Routing(
        torch.zeros((x.shape[0], k), dtype=torch.int32), x[:, :k] * 1.0,
        torch.arange(x.shape[0] * k, dtype=torch.int32).view(-1, k), x.sum(1),
        torch.zeros(x.shape[1], dtype=torch.int64), torch.zeros(x.shape[1] + 1, dtype=torch.int64),
        torch.ones(1, dtype=torch.int64), x.sum(0)[:2] * 1.0, True)
    calls = dict(
        ufp4_rmsnorm=lambda x, w, res, eps: M.B.NormOut(
            x * w, x if res is None else x + res, x.sum(1), None, None),
        ufp4_rmsnorm_bwd=lambda dy, h, w, rstd, dh: (
            dy * w + (0 if dh is None else dh), (dy * h).sum(0)),
        ufp4_moe_route=r,
        ufp4_moe_route_bwd=lambda x, r, dg, dl: x * (0 if dg is None else dg.sum())
        + x * (0 if dl is None else dl.sum()),
        ufp4_moe_dispatch=lambda x, s: x.repeat_interleave(s.shape[1], 0),
        ufp4_moe_dispatch_bwd=lambda dxs, s: dxs.view(*s.shape, -1).sum(1),
        ufp4_moe_combine=lambda ys, s, g, res: (
            (ys.view(*s.shape, -1) * g[:, :, None]).sum(1) + (0 if res is None else res)),
        ufp4_moe_combine_bwd=lambda dy, ys, s, g: (
            (dy[:, None] * g[:, :, None]).reshape(ys.shape),
            (dy[:, None] * ys.view(*s.shape, -1)).sum(2)))
    for name, call in calls.items():
        monkeypatch.setattr(M.B, name, call)


def leaf(*shape):
    return (torch.arange(torch.Size(shape).numel(), dtype=torch.float32).reshape(shape) / 7
            - 0.5).requires_grad_()


def losses_of(x):
    """name: (the loss of a layer's outputs, the tensor to differentiate by)."""
    norm = M.RMSNorm(4, dtype=torch.float32)
    router = M.MoERouter(4, 6, 2, dtype=torch.float32)
    slots = torch.arange(6, dtype=torch.int32).view(3, 2)
    gates, ys = leaf(3, 2), leaf(6, 4)
    y, h = norm(x, leaf(3, 4))
    r = router(x)
    return {"norm": (norm(x).sum(), x), "norm, squared": ((y + h).square().sum(), x),
            "norm's weight": (y.sum(), norm.weight), "gates": (r.gates.sum(), x),
            "losses": (r.losses.square().sum(), router.weight),
            "dispatch": (M.dispatch(x, slots).square().sum(), x),
            "combine": (M.combine(ys, slots, gates).sum(), ys),
            "combine's gates": (M.combine(ys, slots, gates, x).sum(), gates)}


def test_second_derivatives_are_refused(plain):
    """They would be without the layer's part.  The first ones may be part of a
    recorded graph."""
    for name in losses_of(leaf(3, 4)):
        loss, at = losses_of(leaf(3, 4))[name]
        want, = torch.autograd.grad(loss, at, retain_graph=True)
        got, = torch.autograd.grad(loss, at, create_graph=True)
        assert torch.equal(got, want), name
        with pytest.raises(RuntimeError, match="second derivative"):
            (got.square().sum() + at.square().sum()).backward()


def test_gradients_that_are_constant_or_exact_are_not_refused(plain):
    x, slots = leaf(3, 4), torch.arange(6, dtype=torch.int32).view(3, 2)
    # dispatch is linear: the gradient of a sum depends on nothing
    g, = torch.autograd.grad(M.dispatch(x, slots).sum(), x, create_graph=True)
    ((g * x).sum() + x.sum()).backward()
    assert torch.equal(x.grad, g + 1)
    # the residual's gradient is dy itself, the stream's is dh itself
    for stream in (lambda v: M.combine(leaf(6, 4).detach(), slots, leaf(3, 2).detach(), v),
                   lambda v: M.RMSNorm(4, dtype=torch.float32)(leaf(3, 4).detach(), v)[1]):
        x = leaf(3, 4)
        g, = torch.autograd.grad(stream(x).square().sum() / 2, x, create_graph=True)
        g.sum().backward()
        assert torch.equal(x.grad, torch.ones((3, 4)))


def test_a_gradient_that_is_listed_twice_is_clipped_once(monkeypatch):
    """Scaled by two workgroups at once, its elements would be scaled once or
    twice, whichever came first."""
    seen = []
    monkeypatch.setattr(M.B, "ufp4_clip_grads", lambda grads, *a, **kw: seen.extend(grads))
    a, b, c = (torch.nn.Parameter(torch.zeros(3)) for _ in range(3))
    a.grad, b.grad = torch.ones(3), torch.ones(3)
    c.grad = b.grad                                  # two parameters, one gradient
    M.clip_grad_norm_([a, b, a, c, torch.nn.Parameter(torch.zeros(3))], 1.0)
    assert [id(g) for g in seen] == [id(a.grad), id(b.grad)]
