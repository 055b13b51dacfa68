"""Dropout against the oracle, bit for bit: the mask is a function of the seed,
the offset, the row and the column, and the FP32 operations are the oracle's."""
import numpy as np
import pytest
import torch

from oracle import ffn_oracle as O
from uniform_grid_fp4_amd import ffn as F

pytestmark = pytest.mark.gpu
DEV = "cuda"
BOTH = [torch.bfloat16, torch.float32]


def values(t):
    return t.detach().cpu().float().numpy()


def inputs(rows, cols, dtype, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + rows * 7919 + cols)
    n = lambda std: torch.empty((rows, cols), device=DEV).normal_(0.0, std, generator=g).to(dtype)
    return n(1.0), n(2.0)


def check(x, p, seed, offset, res, got):
    want = O.dropout(values(x), p, seed, offset, None if res is None else values(res),
                     x.dtype == torch.bfloat16)
    assert got.dtype == x.dtype and np.array_equal(values(got), want)


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 9), (2, 10), (2, 11), (2, 12), (2, 13), (2, 14), (2, 15),
          (1, 2048), (257, 1411), (64, 6144), (1000, 33), (70000, 1), (3, 40001)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", BOTH)
def test_values(rows, cols, dtype):
    x, res = inputs(rows, cols, dtype)
    for p, seed, offset in ((0.1, 1234567890123456789, 0), (0.5, 3, 2 ** 63 + 5)):
        check(x, p, seed, offset, None, F.ufp4_dropout(x, p, seed, offset))
        check(x, p, seed, offset, res, F.ufp4_dropout(x, p, seed, offset, residual=res))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("p", [0.0, 1.0, 2.0 ** -18, 1 - 2.0 ** -18, 2.0 ** -17, 0.999, 1.0 / 3.0])
def test_probabilities(dtype, p):
    x, res = inputs(300, 70, dtype)
    y = F.ufp4_dropout(x, p, 5, 6, residual=res)
    check(x, p, 5, 6, res, y)
    if p == 0.0:
        assert torch.equal(F.ufp4_dropout(x, p, 5), x)
    if p == 1.0:
        assert torch.equal(y, res) and not F.ufp4_dropout(x, p, 5).any()


def test_seeds_and_offsets():
    """Python integers of any size stand for their 64 bits; an offset on the
    GPU for the same number; other words give other masks."""
    x = torch.ones((40, 100), device=DEV)
    base = F.ufp4_dropout(x, 0.5, 11, 3)
    assert torch.equal(base, F.ufp4_dropout(x, 0.5, 11 + 2 ** 64, 3 - 2 ** 64))
    there = torch.tensor([3], device=DEV)
    assert torch.equal(base, F.ufp4_dropout(x, 0.5, 11, there))
    assert torch.equal(F.ufp4_dropout(x, 0.5, -1, -2), F.ufp4_dropout(x, 0.5, 2 ** 64 - 1, torch.tensor(-2, device=DEV)))
    others = [F.ufp4_dropout(x, 0.5, s, o) for s, o in
              ((12, 3), (11 + 2 ** 32, 3), (11, 4), (11, 3 + 2 ** 32))]
    for y in others:
        assert 0.4 < float((y != base).float().mean()) < 0.6


@pytest.mark.parametrize("dtype", BOTH)
def test_what_is_dropped_is_zero_whatever_it_held(dtype):
    x, res = inputs(20, 64, dtype)
    keep = torch.from_numpy(O.dropout_keep(20, 64, 0.5, 9, 1)).to(DEV)
    x[~keep] = float("nan")
    x[::2][~keep[::2]] = float("inf")
    y = F.ufp4_dropout(x, 0.5, 9, 1)
    assert not y[~keep].any() and y[keep].isfinite().all()
    y = F.ufp4_dropout(x, 0.5, 9, 1, residual=res)
    assert torch.equal(y[~keep], res[~keep])
    x[keep] = float("nan")
    assert F.ufp4_dropout(x, 0.5, 9, 1)[keep].isnan().all()


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("cols,ld,start", [(64, 65, 1), (1001, 1100, 3), (13, 13, 5), (2048, 4096, 0)])
def test_strides_and_in_place(dtype, cols, ld, start):
    x, res = inputs(33, cols, dtype)
    want = F.ufp4_dropout(x, 0.3, 21, 1, residual=res)
    check(x, 0.3, 21, 1, res, want)
    views = []
    for t in (x, res):
        flat = torch.full((start + 33 * ld + 9,), float("nan"), dtype=dtype, device=DEV)
        v = flat[start:start + 33 * ld].view(33, ld)[:, :cols]
        v.copy_(t)
        views.append(v)
    assert torch.equal(F.ufp4_dropout(views[0], 0.3, 21, 1, residual=views[1]), want)
    for into in (0, 1):
        pair = [x.clone(), res.clone()]
        before = pair[into]._version
        got = F.ufp4_dropout(pair[0], 0.3, 21, 1, residual=pair[1], out=pair[into])
        assert got.data_ptr() == pair[into].data_ptr() and pair[into]._version > before
        assert torch.equal(got, want)


def test_backward_is_the_same_call():
    """<dropout(x), dy> = <x, dropout(dy)> up to the products' roundings (FP32,
    three of them on either side), and a difference of two outputs is the
    output of the difference."""
    x, dy = inputs(200, 300, torch.float32)
    y, dx = F.ufp4_dropout(x, 0.25, 8, 2), F.ufp4_dropout(dy, 0.25, 8, 2)
    a, b = (y.double() * dy.double()), (x.double() * dx.double())
    assert ((a - b).abs() <= 4 * 2.0 ** -24 * a.abs()).all() and (y == 0).eq(dx == 0).all()
    d = 2.0 ** -8 * torch.sign(dy)
    up = F.ufp4_dropout(x.sign() + d, 0.25, 8, 2) - F.ufp4_dropout(x.sign(), 0.25, 8, 2)
    # sign(x) + d is exact, its product with the scale rounded
    assert ((up - F.ufp4_dropout(d, 0.25, 8, 2)).abs() <= 4 * 2.0 ** -24).all()


def test_rows_beyond_one_turn_of_the_grid():
    """2^25 elements in rows of 8: the grid's loop, and the row numbers of the
    later turns."""
    rows = 1 << 22
    x = torch.ones((rows, 8), dtype=torch.bfloat16, device=DEV)
    y = F.ufp4_dropout(x, 0.5, 77, 0)
    for row0 in (0, 65536 * 256 // 8, rows - 500):
        keep = O.dropout_keep(500, 8, 0.5, 77, 0, row0=row0)
        assert np.array_equal(values(y[row0:row0 + 500]) != 0, keep)
    # more groups than one turn of 65536 workgroups takes
    x = torch.ones((1, 1 << 24), dtype=torch.bfloat16, device=DEV).expand(12, -1)
    y = F.ufp4_dropout(x.contiguous(), 0.5, 78, 0)
    keep = O.dropout_keep(1, 1 << 24, 0.5, 78, 0, row0=11)
    assert np.array_equal(values(y[11:]) != 0, keep)


def test_captured_call_draws_by_the_offset_on_the_gpu():
    x, res = inputs(300, 256, torch.bfloat16)
    step = torch.zeros((1,), dtype=torch.int64, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        F.ufp4_dropout(x, 0.2, 4, step, residual=res)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = F.ufp4_dropout(x, 0.2, 4, step, residual=res)
    for i in range(4):
        step.fill_(100 + i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, F.ufp4_dropout(x, 0.2, 4, 100 + i, residual=res)), i


def test_no_rows_and_refusals():
    assert F.ufp4_dropout(torch.empty((0, 5), device=DEV), 0.5, 1).shape == (0, 5)
    x, res = inputs(4, 64, torch.bfloat16)
    for call in (lambda: F.ufp4_dropout(x, -0.1, 0), lambda: F.ufp4_dropout(x, 1.1, 0),
                 lambda: F.ufp4_dropout(x, float("nan"), 0), lambda: F.ufp4_dropout(x[0], 0.1, 0),
                 lambda: F.ufp4_dropout(x, 0.1, 0, residual=res[:2]),
                 lambda: F.ufp4_dropout(x, 0.1, 0, residual=res.cpu()),
                 lambda: F.ufp4_dropout(x, 0.1, 0, out=res[:, :32]),
                 lambda: F.ufp4_dropout(x, 0.1, 0, torch.zeros(2, dtype=torch.int64, device=DEV)),
                 lambda: F.ufp4_dropout(x, 0.1, 0, torch.zeros(1, dtype=torch.int64)),
                 lambda: F.ufp4_dropout(x.t(), 0.1, 0)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: F.ufp4_dropout(x, 0.1, 0, residual=res.float()),
                 lambda: F.ufp4_dropout(x, 0.1, 0, torch.zeros(1, device=DEV)),
                 lambda: F.ufp4_dropout(x, 0.1, 0, out=res.float())):
        with pytest.raises(TypeError):
            call()
