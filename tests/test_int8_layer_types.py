"""The int8 layers when a model is cast, moved or loaded, without a GPU."""
import copy

import pytest
import torch

from uniform_grid_fp4_amd import feedforward as W


@pytest.fixture
def layer(monkeypatch):
    monkeypatch.setattr(W.F, "ufp4_int8_quantize", lambda w: W.F.Int8Rows(
        torch.arange(w.shape[0] * 128, dtype=torch.int8).reshape(-1, 128),
        torch.rand(w.shape[0]) + 0.1, w.shape[1]))
    return W.Int8Linear(torch.zeros(6, 20), torch.rand(6))


@pytest.mark.parametrize("cast", [lambda m: m.to(torch.bfloat16), lambda m: m.half(),
                                  lambda m: m.double(), lambda m: m.bfloat16().float(),
                                  lambda m: m.to("cpu", torch.bfloat16)])
def test_scales_stay_what_they_are(layer, cast):
    """The library takes FP32 scales and biases; codes are of no other type."""
    want = copy.deepcopy(layer)
    model = torch.nn.ModuleList([layer, torch.nn.Linear(2, 2)])
    cast(model)
    for name in ("q", "scale", "bias"):
        got, had = getattr(layer, name), getattr(want, name)
        assert got.dtype == had.dtype and torch.equal(got, had)


def test_without_a_bias(layer):
    bare = W.Int8Linear(torch.zeros(6, 20))
    scale = bare.scale.clone()
    bare.half()
    assert bare.bias is None and torch.equal(bare.scale, scale)


def test_moves_and_loads(layer):
    there = copy.deepcopy(layer).to("meta", torch.float16)
    assert there.scale.device.type == there.q.device.type == "meta"
    assert there.scale.dtype == there.bias.dtype == torch.float32
    other = W.Int8Linear(torch.ones(6, 20), torch.rand(6))
    other.load_state_dict({k: v.clone() for k, v in layer.state_dict().items()})
    assert torch.equal(other.scale, layer.scale) and torch.equal(other.q, layer.q)
