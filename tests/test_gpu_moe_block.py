"""The MoE block's layers: each autograd function equals the calls it makes,
the block runs forward and backward with padding, its gradients agree with
differences of a plain torch model where quantization is out of the way, and
captured forward calls replay what the eager ones gave."""
import importlib.util
import os

import pytest
import torch

from uniform_grid_fp4_amd import block as B
from uniform_grid_fp4_amd import moe as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def bf(*shape, seed=0, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.empty(shape, device=DEV).normal_(0.0, std, generator=g).to(torch.bfloat16)


def test_norm_layer():
    layer = M.RMSNorm(96, device=DEV)
    x, r = bf(4, 5, 96, seed=1).requires_grad_(), bf(4, 5, 96, seed=2).requires_grad_()
    y, h = layer(x, r)
    dy, dh = bf(4, 5, 96, seed=3), bf(4, 5, 96, seed=4)
    torch.autograd.backward([y, h], [dy, dh])
    n = B.ufp4_rmsnorm(x.detach().reshape(-1, 96), layer.weight.detach(), r.detach().reshape(-1, 96))
    dx, dw = B.ufp4_rmsnorm_bwd(dy.reshape(-1, 96), n.h, layer.weight.detach(), n.rstd,
                                dh.reshape(-1, 96))
    assert torch.equal(y.reshape(-1, 96), n.y) and torch.equal(h.reshape(-1, 96), n.h)
    assert torch.equal(x.grad.reshape(-1, 96), dx) and torch.equal(r.grad, x.grad)
    assert torch.equal(layer.weight.grad, dw)
    # without a residual, and the stream alone
    layer(x).sum().backward()
    x.grad = r.grad = None
    layer(x, r)[1].backward(dh)
    assert torch.equal(x.grad, dh) and torch.equal(r.grad, dh)
    q = layer.quantized(x, r)
    assert q.y is None and q.q.dtype == torch.float8_e4m3fn
    err = (q.q.float() * q.scale[:, None] - n.y.float()).abs()
    # half an E4M3 step of y, or of the smallest number, and half a bf16 step
    lim = (2.0 ** -4 + 2.0 ** -7) * n.y.float().abs() + q.scale[:, None] * 2.0 ** -9
    assert (err <= lim).all()


def test_broadcast_gradients():
    """Gradients that arrive broadcast (of a sum over everything, and of one
    over the rows) equal the same gradients written out."""
    layer = M.RMSNorm(64, device=DEV)
    slots = B.ufp4_moe_route(bf(6, 8, seed=3), 2).slots
    gates = torch.rand((6, 2), device=DEV)
    for grad in (torch.ones((), dtype=torch.bfloat16, device=DEV).expand(6, 64),
                 bf(64, seed=4).expand(6, 64), bf(6, 1, seed=5).expand(6, 64)):
        got = []
        for dy in (grad, grad.contiguous()):
            x, r = bf(6, 64, seed=1).requires_grad_(), bf(6, 64, seed=2).requires_grad_()
            layer.weight.grad = None
            y, h = layer(x, r)
            xs = M.dispatch(y, slots)
            out = M.combine(xs, slots, gates, h)
            torch.autograd.backward([out, h], [dy, dy])
            got.append([x.grad, r.grad, layer.weight.grad])
        for a, b in zip(*got):
            assert torch.equal(a, b)


def test_router_and_exchange_layers():
    x, valid = bf(70, 64, seed=5).requires_grad_(), torch.arange(70, device=DEV) < 60
    router = M.MoERouter(64, 12, 3, device=DEV)
    r = router(x, valid)
    assert r.gates.requires_grad and r.losses.requires_grad and not r.slots.requires_grad
    xs = M.dispatch(x, r.slots)
    y = M.combine(xs * 2, r.slots, r.gates, x)
    dy, dl = bf(70, 64, seed=6), torch.tensor([0.5, 0.1], device=DEV)
    torch.autograd.backward([y, r.losses], [dy, dl])
    # the same by hand
    xd, w = x.detach(), router.weight.detach()
    logits = torch.nn.functional.linear(xd, w)
    r2 = B.ufp4_moe_route(logits, 3, valid=valid)
    xs2 = B.ufp4_moe_dispatch(xd, r2.slots)
    assert torch.equal(y, B.ufp4_moe_combine(xs2 * 2, r2.slots, r2.gates, xd))
    dys, dg = B.ufp4_moe_combine_bwd(dy, xs2 * 2, r2.slots, r2.gates)
    dlog = B.ufp4_moe_route_bwd(logits, r2, dg, dl)
    assert torch.allclose(router.weight.grad.float(), dlog.float().t() @ xd.float(), atol=2e-2,
                          rtol=2e-2)
    dx = (dy.float() + B.ufp4_moe_dispatch_bwd(dys * 2, r2.slots).float()
          + dlog.float() @ w.float())
    # three bf16 terms, each rounded, and the two sums of them: five half steps
    size = dy.float().abs() + B.ufp4_moe_dispatch_bwd(dys.abs() * 2, r2.slots).float() \
        + dlog.float().abs() @ w.float().abs()
    assert ((x.grad.float() - dx).abs() <= 5 * 2.0 ** -8 * size + 1e-6).all()


def test_block_trains_and_padding_stays_out():
    torch.manual_seed(0)
    block = M.UFP4MoEBlock(128, 96, 8, 2, seed=1, device=DEV)
    x, r = bf(3, 40, 128, seed=7).requires_grad_(), bf(3, 40, 128, seed=8).requires_grad_()
    valid = torch.ones((3, 40), dtype=torch.bool, device=DEV)
    valid[2, 10:] = False
    out = block(x, r, valid)
    assert out.y.shape == x.shape and int(out.counts.sum()) == int(valid.sum()) * 2
    assert not out.y[~valid].any()
    (out.y.float().square().sum() + out.losses.sum()).backward()
    assert not x.grad[~valid].any() and x.grad[valid].any() and torch.equal(x.grad, r.grad)
    for p in block.parameters():
        assert p.grad is not None and p.grad.float().isfinite().all()
    before = [p.grad.float() for p in block.parameters()]
    norm = M.clip_grad_norm_(block.parameters(), 0.5)
    want = torch.stack([g.double().square().sum() for g in before]).sum().sqrt()
    assert abs(float(norm) - float(want)) <= 1e-6 * float(want)
    coef = min(1.0, 0.5 / (float(want) + 1e-6))
    for g, p in zip(before, block.parameters()):
        assert ((p.grad.float() - g * coef).abs() <= 2.0 ** -8 * (g * coef).abs() * 1.01).all()
    # what the padding holds does not matter
    x2 = x.detach().clone()
    x2[~valid] = 100.0
    s0 = block.up.sr_seed
    again = block(x2, r.detach(), valid)
    assert torch.equal(again.y[valid], out.y[valid]) and block.up.sr_seed != s0


def test_captured_calls_replay():
    """Norm, router, dispatch, combine, their backwards and the clip, captured
    once and replayed with eager work between the replays."""
    x, res, w = bf(300, 256, seed=1), bf(300, 256, seed=2), bf(256, seed=3) + 1
    router = bf(16, 256, seed=4, std=0.1)
    grads = [bf(1000, 33, seed=5), bf(77, seed=6).float()]
    outs = [torch.empty_like(g) for g in grads]
    dl = torch.tensor([0.1, 0.01], device=DEV)

    def step():
        n = B.ufp4_rmsnorm(x, w, res, q8=True)
        logits = n.y @ router.t()
        r = B.ufp4_moe_route(logits, 4)
        xs = B.ufp4_moe_dispatch(n.y, r.slots)
        y = B.ufp4_moe_combine(xs, r.slots, r.gates, n.h)
        dys, dg = B.ufp4_moe_combine_bwd(y, xs, r.slots, r.gates)
        dlog = B.ufp4_moe_route_bwd(logits, r, dg, dl)
        dx = B.ufp4_moe_dispatch_bwd(dys, r.slots)
        dxn, dw = B.ufp4_rmsnorm_bwd(dx, n.h, w, n.rstd, y)
        norm = B.ufp4_clip_grads(grads, 0.1, out=outs)
        return [n.y, n.q.view(torch.uint8), r.slots, r.offsets, r.losses, xs, y, dys, dg, dlog,
                dxn, dw, norm, *outs]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(4):
        x.copy_(bf(300, 256, seed=20 + i))
        grads[0].copy_(bf(1000, 33, seed=40 + i))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


def test_another_stream_than_the_default():
    x, w = bf(500, 512, seed=1), bf(512, seed=2)
    want = B.ufp4_rmsnorm(x, w, q8=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = B.ufp4_rmsnorm(x, w, q8=True)
        r = B.ufp4_moe_route(got.y[:, :64].contiguous(), 4)
    side.synchronize()
    assert torch.equal(got.y, want.y) and int(r.counts.sum()) == 2000


def test_example_trains_and_serves():
    spec = importlib.util.spec_from_file_location(
        "moe_block_example", os.path.join(ROOT, "examples", "moe_block.py"))
    E = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(E)
    torch.manual_seed(0)
    model = E.Model(256, 128, 8, 2, 2, DEV)
    trace = E.train(model, 12, 512, 256)
    assert all(v == v for v in trace) and trace[-1] < 0.9 * trace[0], trace
    x = bf(1, 256, seed=9)
    with torch.no_grad():
        want = model(x)[0]
    out = E.serve(model, x)
    assert out.shape == (1, 256)
    # E4M3 rounds a value by 2^-4 of itself or 2^-10 of the row's scale times
    # 448; the projection is the identity and adds bf16 half steps
    lim = (2.0 ** -4 + 2.0 ** -6) * want.float().abs() + want.float().abs().max() * 2.0 ** -17
    assert ((out.float() - want.float()).abs() <= lim).all()
