"""The device that is current while the library is called: the tensors' own.  A
default stream's handle is 0 on every device, which stands for the current
device's, so a call with another one current would launch on the wrong GPU.
Stand-ins for torch's device functions; no GPU needed."""
import contextlib
import types

import pytest
import torch

from uniform_grid_fp4_amd import block as B
from uniform_grid_fp4_amd import ufp4 as U


@pytest.fixture
def current(monkeypatch):
    """[the current device's index], as torch would keep it."""
    at = [0]

    @contextlib.contextmanager
    def device(d):
        before, at[0] = at[0], d.index
        try:
            yield
        finally:
            at[0] = before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: at[0])
    monkeypatch.setattr(B, "_current_device", lambda: at[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    return at


@pytest.mark.parametrize("module", [U, B])
@pytest.mark.parametrize("index", [0, 1, 3])
def test_the_tensors_device_is_current(monkeypatch, current, module, index):
    seen = []

    def some_call(*args):
        seen.append((current[0], args))
        return -1 if args[0] == "refuse" else 0

    monkeypatch.setattr(module, "lib", lambda: types.SimpleNamespace(some_call=some_call))
    monkeypatch.setattr(U, "_stream", lambda d: ("stream of", d.index))
    monkeypatch.setattr(B, "_raw_stream", lambda index: ("stream of", index))
    dev = torch.device("cuda", index)
    module._call("some_call", dev, 1, 2)
    assert seen == [(index, (1, 2, ("stream of", index)))] and current == [0]
    with pytest.raises(U.UFP4Error, match="some_call: UFP4_ERR_INVALID_ARG"):
        module._call("some_call", dev, "refuse")
    assert current == [0]


def test_every_call_with_a_stream_goes_that_way():
    for module in (U, B):
        src = open(module.__file__).read()
        names = [n for n in module.EXPORTS if not n.endswith(("_size", "_string"))]
        for name in names:
            assert f'_call("{name}", ' in src or f'_dense("{name}", ' in src, name
            assert f"lib().{name}(" not in src, name
