"""The masks that the dropout layers draw, on the GPU."""
import pytest
import torch
import torch.utils.checkpoint

from uniform_grid_fp4_amd import feedforward as W
from uniform_grid_fp4_amd import ufp4 as U

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ones(*shape):
    return torch.ones(shape, dtype=torch.bfloat16, device=DEV)


def test_layers_of_a_stack_drop_other_elements():
    """Each keeps half of 65536 elements, any two together a quarter: 6 standard
    deviations of a share of 1/4."""
    drops = [W.UFP4FeedForward(64, 64, p=0.5, device=DEV).drop for _ in range(4)]
    kept = [d(ones(256, 256)).bool() for d in drops]
    for i in range(4):
        for j in range(i):
            share = float((kept[i] & kept[j]).double().mean())
            assert abs(share - 0.25) < 6 * (0.1875 / 65536) ** 0.5


def bf(*shape, seed=0, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.empty(shape, device=DEV).normal_(0.0, std, generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("reentrant", [False, True])
@pytest.mark.parametrize("there", [False, True])
def test_recomputed_sublayers_have_the_gradients_of_plain_ones(reentrant, there):
    """Two sublayers in one recomputed region, so that the second's input is that of
    the first's mask; dY rounded to nearest, whose noise would differ."""
    torch.manual_seed(0)
    layers = [W.UFP4FeedForward(128, 192, p=0.3, device=DEV) for _ in range(2)]
    for layer in layers:
        layer.gated.rnd_dy = layer.down.rnd_dy = U.ROUND_RTNE
    offset = torch.tensor([11], device=DEV) if there else 11
    x, dy = bf(50, 128, seed=1).requires_grad_(), bf(50, 128, seed=2)
    leaves = [x, *(p for layer in layers for p in layer.parameters())]

    def run(t):
        return layers[1](layers[0](t, offset=offset), offset=offset)

    y = run(x)
    want = torch.autograd.grad(y, leaves, dy)
    again = torch.utils.checkpoint.checkpoint(run, x, use_reentrant=reentrant)
    assert torch.equal(again, y)
    again.backward(dy)
    for p, g in zip(leaves, want):
        assert torch.equal(p.grad, g)


def test_a_captured_sublayer_draws_by_its_offset():
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    layer = W.UFP4FeedForward(128, 192, p=0.3, device=DEV, offset=step)
    x, r = bf(70, 128, seed=1), bf(70, 128, seed=2)
    with torch.no_grad():
        layer(x, r)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = layer(x, r)
        seen = []
        for i in range(4):
            step.fill_(20 + i)
            x.copy_(bf(70, 128, seed=1))
            graph.replay()
            torch.cuda.synchronize()
            seen.append(y.clone())
            assert torch.equal(seen[-1], layer(x, r, offset=20 + i)), i
    assert layer.drop.calls == 0
    assert not any(torch.equal(seen[i], seen[j]) for i in range(4) for j in range(i))
