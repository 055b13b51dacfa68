"""The int8 product of a few rows to many columns, whose rows are quantized into a
workspace where there is one: bit for bit the two calls it stands for, with the
binding's workspace, the caller's, and none."""
import pytest
import torch

from test_gpu_ffn_int8 import BOTH, normal
from uniform_grid_fp4_amd import ffn as F

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("m,k", [(1, 130), (1, 2048), (2, 700), (5, 64), (16, 1024), (16, 3)])
@pytest.mark.parametrize("dtype", BOTH)
def test_wide(m, k, dtype):
    f = F.INT8_FEW_COLUMNS + 21
    x, w = normal(m, k, dtype), F.ufp4_int8_quantize(normal(2 * f, k, seed=2, std=0.05))
    bias = normal(1, 2 * f, seed=3)[0].contiguous()
    assert F.ufp4_int8_linear_workspace_size(m, k) == 0
    for kw in (dict(), dict(bias=bias, act=F.ACT_SILU), dict(act=F.ACT_GELU)):
        want = F.ufp4_int8_gemm(F.ufp4_int8_quantize(x), w, out_dtype=dtype, **kw)
        own = torch.empty(F.ufp4_int8_linear_workspace_size(m, k, True), dtype=torch.uint8,
                          device=DEV)
        for ws in (None, own, own[:0]):
            assert torch.equal(F.ufp4_int8_linear(x, w, workspace=ws, **kw), want)
    none = torch.empty((0, k), dtype=dtype, device=DEV)
    assert F.ufp4_int8_linear(none, w).shape == (0, 2 * f)


def test_captured():
    """The workspace of a captured call is the graph's own."""
    w = F.ufp4_int8_quantize(normal(20000, 256, seed=2, std=0.05))
    x = normal(4, 256, torch.bfloat16)
    F.ufp4_int8_linear(x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = F.ufp4_int8_linear(x, w)
    for i in range(4):
        x.copy_(normal(4, 256, torch.bfloat16, seed=10 + i))
        want = F.ufp4_int8_linear(x, w)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
