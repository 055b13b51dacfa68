"""The feed-forward layers: each autograd function equals the calls it makes, the
sublayer and the gated MoE block run forward and backward, what is served in int8
stays within the codes' half steps, captured calls replay what the eager ones
gave, and the example runs."""
import importlib.util
import os

import pytest
import torch

from uniform_grid_fp4_amd import block as B
from uniform_grid_fp4_amd import feedforward as W
from uniform_grid_fp4_amd import ffn as F
from uniform_grid_fp4_amd import moe as M
from uniform_grid_fp4_amd import ufp4 as U

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def bf(*shape, seed=0, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.empty(shape, device=DEV).normal_(0.0, std, generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("bias", [True, False])
def test_layer_norm(bias):
    layer = W.LayerNorm(96, bias=bias, device=DEV)
    x, r = bf(4, 5, 96, seed=1).requires_grad_(), bf(4, 5, 96, seed=2).requires_grad_()
    y, h = layer(x, r)
    dy, dh = bf(4, 5, 96, seed=3), bf(4, 5, 96, seed=4)
    torch.autograd.backward([y, h], [dy, dh])
    w, b = layer.weight.detach(), layer.bias.detach() if bias else None
    n = F.ufp4_layernorm(x.detach().reshape(-1, 96), w, b, r.detach().reshape(-1, 96))
    dx, dw, db = F.ufp4_layernorm_bwd(dy.reshape(-1, 96), n.h, w, n.mean, n.rstd,
                                      dh.reshape(-1, 96), bias=bias)
    assert torch.equal(y.reshape(-1, 96), n.y) and torch.equal(h.reshape(-1, 96), n.h)
    assert torch.equal(x.grad.reshape(-1, 96), dx) and torch.equal(r.grad, x.grad)
    assert torch.equal(layer.weight.grad, dw)
    assert not bias or torch.equal(layer.bias.grad, db)
    # a broadcast gradient equals the same written out
    got = []
    for d in (torch.ones((), dtype=torch.bfloat16, device=DEV).expand(4, 5, 96),
              torch.ones((4, 5, 96), dtype=torch.bfloat16, device=DEV)):
        x.grad = None
        layer(x).backward(d)
        got.append(x.grad)
    assert torch.equal(*got)


def test_dropout_layer():
    drop = W.Dropout(0.3, seed=9)
    x, r = bf(6, 7, 80, seed=1).requires_grad_(), bf(6, 7, 80, seed=2).requires_grad_()
    y = drop(x, r)
    dy = bf(6, 7, 80, seed=3)
    y.backward(dy)
    flat = lambda t: t.detach().reshape(-1, 80)
    assert torch.equal(flat(y), F.ufp4_dropout(flat(x), 0.3, 9, 1, residual=flat(r)))
    assert torch.equal(flat(x.grad), F.ufp4_dropout(flat(dy), 0.3, 9, 1))
    assert torch.equal(r.grad, dy)
    assert not torch.equal(drop(x, r), y)
    drop.eval()
    assert drop(x) is x and torch.equal(drop(x, r), (x.float() + r.float()).to(torch.bfloat16))
    # the gradient of a sum arrives broadcast
    x.grad = None
    W.dropout(x, 0.5, 1).sum().backward()
    assert torch.equal(flat(x.grad), F.ufp4_dropout(torch.ones_like(flat(x)), 0.5, 1))


@pytest.mark.parametrize("experts", [0, 3])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_layers_are_their_calls(experts, act):
    t, k, f = 150, 96, 70
    if experts:
        layer = W.UFP4GatedExpertLinear(experts, k, f, act=act, seed=3, device=DEV)
        offsets = torch.tensor([0, 50, 50, 150], device=DEV)
        more, how = (offsets,), dict(col_axis=U.BLOCKS_ALONG_ROWS_STACKED, n_groups=experts)
    else:
        layer = W.UFP4GatedLinear(k, f, act=act, seed=3, device=DEV)
        offsets, more, how = None, (), {}
    x, dy = bf(t, k, seed=1).requires_grad_(), bf(t, f, seed=2, std=1e-2)
    y = layer(x, *more)
    y.backward(dy)
    mf, md, mw = layer.masks
    xq, xtq = U.ufp4_rht_quantize_dual(x.detach(), (True, mf, 0), (True, mw, 0),
                                       group_offsets=offsets)
    wq, wtq = U.ufp4_rht_quantize_dual(layer.weight.detach(), (True, mf, 0), (True, md, 0), **how)
    out = F.ufp4_gated_gemm(xq, wq, layer.act, offsets=offsets)
    assert torch.equal(y, out.y)
    dgu = F.ufp4_gated_bwd(dy, out.gu, layer.act)
    dq, dtq = U.ufp4_rht_quantize_dual(dgu, (True, md, 0), (True, mw, 1), rnd=U.ROUND_SR,
                                       seed=layer.sr_seed, group_offsets=offsets)
    if experts:
        dx = U.ufp4_grouped_gemm_out(U.DGRAD, offsets, dq, wtq)
        dw = U.ufp4_grouped_gemm_out(U.WGRAD, offsets, dtq, xtq).reshape(-1, k)
    else:
        dx, dw = U.ufp4_gemm_out(U.DGRAD, dq, wtq), U.ufp4_gemm_out(U.WGRAD, dtq, xtq)
    assert torch.equal(x.grad, dx) and torch.equal(layer.weight.grad, dw)


def test_gated_gradients_follow_the_formula():
    """Against the gradients in 64 bits of the product of the unquantized operands.
    A 4-bit operand is off by up to 1/14 of its block's largest element; over the
    two operands of each GEMM and the three GEMMs on the way the errors add up to
    a few tenths of a gradient's norm at most, and they are not along it."""
    t, k, f = 512, 256, 320
    layer = W.UFP4GatedLinear(k, f, seed=1, device=DEV)
    x, dy = bf(t, k, seed=1).requires_grad_(), bf(t, f, seed=2)
    layer(x).backward(dy)
    x2 = x.detach().double().requires_grad_()
    w2 = layer.weight.detach().double().requires_grad_()
    gu = x2 @ w2.t()
    (torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]).backward(dy.double())
    for got, want in ((x.grad, x2.grad), (layer.weight.grad, w2.grad)):
        off = (got.double() - want).norm() / want.norm()
        along = (got.double() * want).sum() / want.square().sum()
        assert off < 0.4 and abs(along - 1) < 0.1, (float(off), float(along))


def test_sublayer_trains_and_repeats():
    """Forward and backward of the whole, equal to its layers one by one."""
    torch.manual_seed(0)
    block = W.UFP4FeedForward(128, 192, p=0.2, seed=4, device=DEV)
    x, r = bf(3, 40, 128, seed=7).requires_grad_(), bf(3, 40, 128, seed=8).requires_grad_()
    out = block(x, r)
    seeds = block.gated.sr_seed, block.down.sr_seed, block.drop.calls
    dy = bf(3, 40, 128, seed=9)
    out.backward(dy)
    grads = [p.grad.clone() for p in (x, r, *block.parameters())]
    assert all(g.float().isfinite().all() and g.any() for g in grads)
    assert torch.equal(grads[0], grads[1])
    # the same step again, by hand
    for p in (x, r, *block.parameters()):
        p.grad = None
    block.gated.sr_seed, block.down.sr_seed = seeds[0] - 1, seeds[1] - 1
    y, h = block.norm(x, r)
    again = W.dropout(block.down(block.gated(y)), 0.2, 4, seeds[2], h)
    again.backward(dy)
    assert torch.equal(again, out)
    for g, p in zip(grads, (x, r, *block.parameters())):
        assert torch.equal(g, p.grad)
    block.eval()
    assert torch.equal(block.drop(x, r), (x.float() + r.float()).to(torch.bfloat16))
    empty = block(x[:, :0].detach(), r[:, :0].detach())
    assert empty.shape == (3, 0, 128)


def test_gated_moe_block():
    torch.manual_seed(0)
    block = M.UFP4MoEBlock(128, 96, 8, 2, seed=1, device=DEV, gated="silu")
    x, r = bf(3, 40, 128, seed=7).requires_grad_(), bf(3, 40, 128, seed=8).requires_grad_()
    valid = torch.ones((3, 40), dtype=torch.bool, device=DEV)
    valid[2, 10:] = False
    out = block(x, r, valid)
    assert out.y.shape == x.shape and not out.y[~valid].any() and out.y[valid].any()
    (out.y.float().square().sum() + out.losses.sum()).backward()
    assert not x.grad[~valid].any() and x.grad[valid].any()
    for p in block.parameters():
        assert p.grad is not None and p.grad.float().isfinite().all() and p.grad.any()
    # what the padding holds does not matter
    x2 = x.detach().clone()
    x2[~valid] = 100.0
    assert torch.equal(block(x2, r.detach(), valid).y[valid], out.y[valid])
    # served: the same routing, the experts' products in int8
    served = W.Int8MoEBlock(block)
    got = served(x.detach(), r.detach(), valid)
    assert torch.equal(got.counts, out.counts) and torch.equal(got.residual, out.residual)
    assert not got.y[~valid].any()
    y, _ = block.norm(x.detach(), r.detach())
    route = block.router(y, valid.reshape(-1))
    xs = M.dispatch(y, route.slots)
    up = F.ufp4_int8_linear(xs, F.ufp4_int8_quantize(block.up.weight.detach()), act=F.ACT_SILU,
                            offsets=route.offsets)
    ys = F.ufp4_int8_linear(up, F.ufp4_int8_quantize(block.down.weight.detach()),
                            offsets=route.offsets)
    want = M.combine(ys, route.slots, route.gates)
    assert torch.equal(got.y.reshape(-1, 128), want)


@pytest.mark.parametrize("t", [1, 200])
def test_int8_linear_within_half_steps(t):
    """Against the exact product: a code is off by half a step and the roundings of
    the quantizer (127 times 2^-22 of a step), so p is off by at most sum |x| sw/2 +
    |w| sx/2 + sx sw/4, a hundredth more, and the output's bf16 half step."""
    x, w = bf(t, 130, seed=1), bf(48, 130, seed=2, std=0.1)
    bias = bf(48, seed=3)
    layer = W.Int8Linear(w, bias)
    y = layer(x.reshape(1, t, 130)).reshape(t, 48)
    xd, wd = x.double(), w.double()
    want = xd @ wd.t() + bias.double()
    sx, sw = xd.abs().amax(1, keepdim=True) / 127, wd.abs().amax(1, keepdim=True) / 127
    lim = xd.abs().sum(1, keepdim=True) @ sw.t() / 2 + sx @ wd.abs().sum(1, keepdim=True).t() / 2 \
        + 130 * sx @ sw.t() / 4
    lim = 1.01 * lim + 2.0 ** -8 * (want.abs() + lim) + 1e-6
    assert ((y.double() - want).abs() <= lim).all()
    with pytest.raises(ValueError):
        layer(x, torch.tensor([0, t], device=DEV))
    with pytest.raises(ValueError):
        W.Int8Linear(w, n_experts=2)(x)


def test_served_sublayer():
    torch.manual_seed(1)
    block = W.UFP4FeedForward(128, 192, p=0.2, seed=4, device=DEV, act="gelu")
    served = W.Int8FeedForward(block)
    for shape in ((1, 128), (2, 70, 128)):
        x, r = bf(*shape, seed=5), bf(*shape, seed=6)
        out = served(x, r)
        y, h = block.norm(x, r)
        flat = lambda t: t.detach().reshape(-1, t.shape[-1])
        a = F.ufp4_int8_linear(flat(y), F.ufp4_int8_quantize(block.gated.weight.detach()),
                               act=F.ACT_GELU)
        b = F.ufp4_int8_linear(a, F.ufp4_int8_quantize(block.down.weight.detach()))
        want = (b.float() + flat(h).float()).to(torch.bfloat16)
        assert out.shape == x.shape and torch.equal(flat(out), want) and not out.requires_grad
        assert torch.equal(served(x), served(x))


def test_captured_calls_replay():
    """All operators captured once, forward and backward, and replayed with eager
    work between the replays."""
    x, res, w, b = bf(300, 256, seed=1), bf(300, 256, seed=2), bf(256, seed=3) + 1, bf(256, seed=4)
    wg, wd = bf(2 * 320, 256, seed=5, std=0.06), bf(256, 320, seed=6, std=0.06)
    w8, d8 = F.ufp4_int8_quantize(wg), F.ufp4_int8_quantize(wd)
    wq = U.ufp4_rht_quantize(wg, U.BLOCKS_ALONG_COLS)
    offsets = torch.tensor([0, 300], device=DEV)
    step_no = torch.zeros(1, dtype=torch.int64, device=DEV)

    def step():
        n = F.ufp4_layernorm(x, w, b, res)
        out = F.ufp4_gated_gemm(U.ufp4_rht_quantize(n.y, U.BLOCKS_ALONG_COLS), wq,
                                offsets=offsets)
        served = F.ufp4_int8_linear(n.y, w8, act=F.ACT_SILU)
        y = F.ufp4_int8_linear(served, d8)
        few = F.ufp4_int8_linear(served[:5], d8, offsets=torch.clamp(offsets, max=5))
        z = F.ufp4_dropout(y, 0.3, 5, step_no, residual=n.h)
        dy = F.ufp4_dropout(z, 0.3, 5, step_no)
        dgu = F.ufp4_gated_bwd(served, out.gu)
        dx, dw, db = F.ufp4_layernorm_bwd(dy, n.h, w, n.mean, n.rstd, z)
        return [*n, *out, served, y, few, z, dy, dgu, dx, dw, db]

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
        step_no.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        want = step()
        torch.cuda.synchronize()
        for j, (p, q) in enumerate(zip(got, want)):
            assert torch.equal(p, q), (i, j)


def test_captured_products_of_every_kind_of_tile():
    """int8 products from one row to the largest tiles, dense and by experts, and the
    gated product of few tiles and of many, in one graph; two graphs of them that
    share nothing replay in turn."""
    shapes = [(1, 256, 4096), (20, 300, 2000), (60, 130, 1000), (200, 512, 1500), (905, 1536, 1411),
              (1000, 2048, 700), (2000, 2050, 900), (2900, 5000, 1411)]
    ws = [F.ufp4_int8_quantize(bf(n, k, seed=i, std=0.05)) for i, (m, n, k) in enumerate(shapes)]
    experts = F.ufp4_int8_quantize(bf(4 * 256, 640, seed=30, std=0.05))
    offsets = torch.tensor([0, 70, 70, 300, 500], device=DEV)
    wq = U.ufp4_rht_quantize(bf(2 * 640, 512, seed=31, std=0.05), U.BLOCKS_ALONG_COLS)

    def inputs(seed):
        return [bf(m, k, seed=seed + i) for i, (m, n, k) in enumerate(shapes)] + \
            [bf(500, 640, seed=seed + 40), bf(40, 512, seed=seed + 41), bf(3000, 512, seed=seed + 42)]

    def step(xs):
        out = [F.ufp4_int8_linear(x, w, act=F.ACT_SILU if w.q.shape[0] % 2 == 0 else F.ACT_NONE)
               for x, w in zip(xs, ws)]
        out.append(F.ufp4_int8_linear(xs[-3], experts, offsets=offsets))
        for x in xs[-2:]:
            out += F.ufp4_gated_gemm(U.ufp4_rht_quantize(x, U.BLOCKS_ALONG_COLS), wq)
        return out

    held = [inputs(100), inputs(200)]
    step(held[0])
    torch.cuda.synchronize()
    graphs, captured = [], []
    for xs in held:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            captured.append(step(xs))
    for i in range(4):
        for x, new in zip(held[i % 2], inputs(300 + 100 * i)):
            x.copy_(new)
        want = step(held[i % 2])
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        for j, (p, q) in enumerate(zip(captured[i % 2], want)):
            assert torch.equal(p, q), (i, j)


def test_two_streams_at_once():
    """The same calls on two streams without waits between them, workspaces of
    their own: what each gives alone."""
    x, w = bf(700, 512, seed=1), bf(512, seed=2)
    w8 = F.ufp4_int8_quantize(bf(640, 512, seed=3))
    other = bf(700, 512, seed=4)

    def work(t):
        n = F.ufp4_layernorm(t, w, w)
        y = F.ufp4_int8_linear(n.y, w8, act=F.ACT_GELU)
        return [n.y, y, *F.ufp4_layernorm_bwd(t, n.h, w, n.mean, n.rstd),
                F.ufp4_dropout(t, 0.5, 1, 2)]

    want = [work(x), work(other)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, t in enumerate((x, other)):
            with torch.cuda.stream(streams[i]):
                got[i].append(work(t))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            for p, q in zip(run, want[i]):
                assert torch.equal(p, q)


def test_block_operators_feed_the_int8_product():
    """The router's offsets go to the grouped int8 product as to the 4-bit ones."""
    x = bf(90, 128, seed=1)
    r = B.ufp4_moe_route(bf(90, 6, seed=2), 2)
    xs = B.ufp4_moe_dispatch(x, r.slots)
    w = bf(6 * 40, 128, seed=3, std=0.1)
    ys = F.ufp4_int8_linear(xs, F.ufp4_int8_quantize(w), offsets=r.offsets)
    for i in (0, 17, 89):
        for j in range(2):
            e, row = int(r.experts[i, j]), int(r.slots[i, j])
            one = F.ufp4_int8_linear(x[i:i + 1], F.ufp4_int8_quantize(w[40 * e:40 * e + 40]))
            assert torch.equal(ys[row], one[0])


def test_example_runs():
    spec = importlib.util.spec_from_file_location(
        "feed_forward_example", os.path.join(ROOT, "examples", "feed_forward.py"))
    E = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(E)
    torch.manual_seed(0)
    model = W.UFP4FeedForward(128, 256, p=0.1, device=DEV)
    trace = E.train(model, 3, 256, 128)
    assert len(trace) == 3 and all(v == v for v in trace)
    assert all(p.grad is not None and p.grad.float().isfinite().all() for p in model.parameters())
    assert W.Int8FeedForward(model)(bf(1, 128, seed=9)).shape == (1, 128)
