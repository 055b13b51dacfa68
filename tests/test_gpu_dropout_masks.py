"""The masks that the dropout layers draw, on the GPU."""
import pytest
import torch

from uniform_grid_fp4_amd import feedforward as W

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
