"""Which masks the dropout layers name, without a GPU: the library's call stands in
as a note of (seed, offset)."""
import copy
import itertools

import pytest
import torch
import torch.utils.checkpoint

from uniform_grid_fp4_amd import feedforward as W
from uniform_grid_fp4_amd import layers as Y


@pytest.fixture
def seen(monkeypatch):
    """(seed, offset) of every call, forward or backward."""
    calls = []

    def call(x, p, seed, offset, residual=None):
        calls.append((seed, int(offset)))
        return x * 0.5 if residual is None else x * 0.5 + residual

    monkeypatch.setattr(W.F, "ufp4_dropout", call)
    return calls


def test_layers_have_masks_of_their_own(seen):
    x = torch.ones(2, 4)
    drops = [W.Dropout(0.5) for _ in range(3)] + [W.UFP4FeedForward(8, 4, p=0.1).drop
                                                  for _ in range(3)]
    drops += [copy.deepcopy(drops[0]), copy.deepcopy(torch.nn.ModuleList([drops[1]]))[0]]
    for d in drops:
        d(x)
    assert len(set(seen)) == len(drops)
    # a run that seeds torch and builds the same layers draws the same
    again = []
    for _ in range(2):
        W._drawn = itertools.count(1)
        torch.manual_seed(7)
        again.append([W.Dropout(0.5).seed, W.UFP4FeedForward(8, 4, p=0.1).drop.seed])
    assert again[0] == again[1] and again[0][0] != again[0][1]
    assert all(0 <= s < 1 << 64 for s in again[0])


def test_a_given_seed_is_kept():
    assert W.Dropout(0.5, seed=3).seed == 3 and W.Dropout(0.5, 0).seed == 0
    layer = W.UFP4FeedForward(8, 4, p=0.1, seed=3)
    assert layer.drop.seed == copy.deepcopy(layer).drop.seed == 3
    assert layer.gated.masks == Y.draw_sign_masks(3) and layer.down.masks == Y.draw_sign_masks(4)


def test_the_products_of_a_layer_without_a_seed_have_zero():
    layer = W.UFP4FeedForward(8, 4)
    assert layer.gated.masks == Y.draw_sign_masks(0) and layer.down.masks == Y.draw_sign_masks(1)
    assert layer.gated.sr_seed == 0 and layer.down.sr_seed == 0x9E3779B97F4A7C15


def test_building_a_layer_draws_nothing_from_torch():
    torch.manual_seed(1)
    before = torch.get_rng_state()
    W.Dropout(0.5)
    assert torch.equal(before, torch.get_rng_state())


def test_a_state_dict_goes_on_with_the_masks(seen):
    x = torch.ones(2, 4)
    for make in (lambda: W.Dropout(0.5), lambda: W.Dropout(0.5, seed=2 ** 64 - 3),
                 lambda: W.Dropout(0.5, seed=-1)):
        old, new = make(), make()
        for _ in range(3):
            old(x)
        new.load_state_dict(old.state_dict())
        del seen[:]
        old(x), new(x)
        word = (1 << 64) - 1
        assert seen[0][0] & word == seen[1][0] & word and seen[0][1] == seen[1][1] == 4
    # as a part of a sublayer, through what only tensors pass
    old, new = W.UFP4FeedForward(8, 4, p=0.5), W.UFP4FeedForward(8, 4, p=0.5)
    old.drop(x)
    state = old.state_dict()
    assert all(isinstance(v, torch.Tensor) for v in state.values())
    new.load_state_dict({k: v.clone() for k, v in state.items()})
    assert (new.drop.seed, new.drop.calls) == (old.drop.seed, 1)


def test_a_state_dict_from_before_loads():
    """Without the masks' place a layer keeps its own."""
    layer = W.UFP4FeedForward(8, 4, p=0.5)
    seed = layer.drop.seed
    layer.drop.calls = 2
    state = {k: v for k, v in layer.state_dict().items() if "drop" not in k}
    assert len(state) == 4
    layer.load_state_dict(state)
    assert (layer.drop.seed, layer.drop.calls) == (seed, 2)
    with pytest.raises(RuntimeError, match="Missing"):
        layer.load_state_dict({k: v for k, v in state.items() if "down" not in k})


def test_recomputed_with_an_offset_in_a_tensor(seen):
    """Recomputation hands what was saved out once."""
    x, step = torch.ones(2, 4, requires_grad=True), torch.tensor([3])
    torch.utils.checkpoint.checkpoint(lambda t: W.dropout(t, 0.5, 1, step).sin(), x,
                                      use_reentrant=False).sum().backward()
    assert set(seen) == {(1, 3)}


def test_a_call_takes_an_offset(seen):
    """In place of the layer's count, and of the layer's own tensor."""
    x = torch.ones(2, 4, requires_grad=True)
    step = torch.tensor([9])
    for drop in (W.Dropout(0.5, seed=1), W.Dropout(0.5, seed=1, offset=step)):
        del seen[:]
        drop(x, offset=5).sum().backward()
        drop(x, x, torch.tensor([6])).sum().backward()
        assert seen == [(1, 5), (1, 5), (1, 6), (1, 6)] and drop.calls == 0
        drop.eval()
        assert drop(x, offset=5) is x


@pytest.mark.parametrize("reentrant", [False, True])
def test_recomputed_calls(seen, reentrant):
    """A call that runs again in the backward pass names the mask it named before,
    or is refused: with the next one the gradients would not be the loss's."""
    x = torch.ones(2, 4, requires_grad=True)
    run = lambda *a: torch.utils.checkpoint.checkpoint(*a, use_reentrant=reentrant).sum()
    drop = W.Dropout(0.5, seed=1)
    run(lambda t: drop(t, None, 5).sin(), x).backward()
    assert {at for _, at in seen} == {5}
    layer = W.Dropout(0.5, seed=1, offset=torch.tensor([6]))
    del seen[:]
    run(lambda t: layer(t).sin(), x).backward()
    assert {at for _, at in seen} == {6}
    loss = run(lambda t: drop(t).sin(), x)
    with pytest.raises(RuntimeError, match="offset"):
        loss.backward()
    assert drop.calls == 1
    drop(x).sum().backward()                     # the next call is none of that
    assert drop.calls == 2
    # nothing is drawn where nothing is dropped
    none = W.Dropout(0.0)
    run(lambda t: none(t, t).sin(), x).backward()


def test_the_sublayer_hands_an_offset_on(seen, monkeypatch):
    layer = W.UFP4FeedForward(8, 4, p=0.5, seed=3, offset=torch.tensor([4]))
    for part in ("norm", "gated", "down"):
        monkeypatch.setattr(layer, part, torch.nn.Identity())
    x = torch.ones(2, 8)
    layer(x), layer(x, offset=8)
    assert seen == [(3, 4), (3, 8)]


def test_the_state_lies_on_the_host_whatever_the_default_device():
    drop = W.Dropout(0.5)
    with torch.device("meta"):
        state = drop.state_dict()
    W.Dropout(0.5).load_state_dict(state)


def test_copies_follow_the_callers_offset(seen):
    """The tensor is the caller's, who advances one; where it is a part of what is
    copied, the copy has the copied one."""
    step = torch.tensor([4])
    layers = [W.UFP4FeedForward(8, 4, p=0.5, offset=step)]
    layers.append(copy.deepcopy(layers[0]))
    assert layers[1].drop.offset is step and layers[1].drop.seed != layers[0].drop.seed
    model = torch.nn.Module()
    model.register_buffer("step", step)
    model.drop = layers[0].drop
    there = copy.deepcopy(model)
    assert there.step is not step and there.drop.offset is there.step
    assert copy.deepcopy(W.Dropout(0.5)).offset is None
