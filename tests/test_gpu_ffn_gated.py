"""The gated product on 4-bit operands, dense and grouped, and its backward.

g and u are those of ufp4_gemm_out (whose own parity with the oracle other tests
show) up to the order of the sums: both add up K / 16 block terms, in a chain or in
eight chains and their sum, so each is within (K / 16 + 8) 2^-24 of the sum of
the terms' sizes, which is at most sum |x| |w|; y and the gradients are checked against the 64-bit
activation of those very FP32 values, within the oracle's error bounds of the
activation, one or two more products' roundings (2^-24 each) and half a step of
the output's type (bf16 2^-8)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import ffn_oracle as O
from oracle import ufp4_oracle as Q
from uniform_grid_fp4_amd import ffn as F
from uniform_grid_fp4_amd import ufp4 as U

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS32 = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: EPS32}
TINY = 1e-36
ACTS = [F.ACT_SILU, F.ACT_GELU]


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def bf(*shape, seed=0, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.empty(shape, device=DEV).normal_(0.0, std, generator=g).to(torch.bfloat16)


def quantized(t, grid=U.GRID_UNIFORM, rht=True, mask=0xACE1):
    return U.ufp4_rht_quantize(t, U.BLOCKS_ALONG_COLS, rht, mask if rht else 0, grid)


def check_y(y, gu, act):
    """y against act(g) * u of FP32 g and u."""
    f = y.shape[1]
    g, u = f64(gu[:, :f]), f64(gu[:, f:])
    value, _ = O.act(g, act)
    err, _ = O.act_error(g, act, EPS32)
    want = value * u
    lim = err * np.abs(u) + 2 * EPS32 * np.abs(want) + HALF[y.dtype] * np.abs(want) * 1.01 + TINY
    assert (np.abs(f64(y) - want) <= lim).all()


def near(got, want, xq, wq, offsets=None):
    """Two sums of the same block terms."""
    x, w = (U.ufp4_dequantize(q).double().abs() for q in (xq, wq))
    if offsets is None:
        size = x @ w.t()
    else:
        at, e = offsets.tolist(), offsets.numel() - 1
        w = w.reshape(e, -1, w.shape[1])
        size = torch.cat([x[a:b] @ w[i].t() for i, (a, b) in enumerate(zip(at[:-1], at[1:]))])
    lim = 2 * (xq.kpad / 16 + 8) * EPS32 * size + TINY
    return bool(((got.double() - want.double()).abs() <= lim).all())


SHAPES = [(1, 16, 1), (1, 2048, 64), (3, 17, 5), (127, 100, 33), (128, 64, 64), (129, 80, 65),
          (257, 1000, 333), (300, 48, 200), (64, 4096, 96), (33, 2050, 40), (2000, 64, 700),
          (500, 100, 8000)]


@pytest.mark.parametrize("t,k,f", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_dense(t, k, f, act):
    x, w = bf(t, k, seed=1), bf(2 * f, k, seed=2, std=2.0 * k ** -0.5)
    xq, wq = quantized(x), quantized(w)
    out = F.ufp4_gated_gemm(xq, wq, act, out_dtype=torch.float32)
    want = U.ufp4_gemm_out(U.FPROP, xq, wq, torch.float32)
    assert near(out.gu, want, xq, wq)
    check_y(out.y, out.gu, act)
    low = F.ufp4_gated_gemm(xq, wq, act)
    assert torch.equal(low.gu, out.gu.to(torch.bfloat16)) and low.y.dtype == torch.bfloat16
    assert torch.equal(low.y, out.y.to(torch.bfloat16))
    lone = F.ufp4_gated_gemm(xq, wq, act, keep=False)
    assert lone.gu is None and torch.equal(lone.y, low.y)


@pytest.mark.parametrize("grid", [U.GRID_UNIFORM, U.GRID_E2M1, U.GRID_E2M1_MAX2])
def test_grids_against_the_oracle(grid):
    """From the quantized operands on, without any other call of the library."""
    t, k, f = 70, 200, 45
    xq, wq = quantized(bf(t, k, seed=3), grid), quantized(bf(2 * f, k, seed=4, std=0.2), grid)
    out = F.ufp4_gated_gemm(xq, wq, F.ACT_SILU, out_dtype=torch.float32)
    c = lambda q: (q.codes.cpu().numpy(), q.scales.cpu().numpy())
    ref, bound = Q.gemm_tn(*c(xq), *c(wq), grid)
    assert (np.abs(f64(out.gu) - ref) <= 1e-5 * bound).all()
    check_y(out.y, out.gu, F.ACT_SILU)


COUNTS = [[5, 0, 130, 1, 0, 64], [700, 0, 1300, 900], [0, 0, 7], [300], [1] * 40, [0, 129]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("act", ACTS)
def test_grouped(counts, act):
    """Each expert's rows with its own weights; empty experts anywhere."""
    e, k, f = len(counts), 96, 70
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    offsets = torch.from_numpy(off).to(DEV)
    x, w = bf(int(off[-1]), k, seed=5), bf(e * 2 * f, k, seed=6, std=0.2)
    xq, wq = quantized(x), quantized(w)
    out = F.ufp4_gated_gemm(xq, wq, act, offsets=offsets, out_dtype=torch.float32)
    want = U.ufp4_grouped_gemm_out(U.FPROP, offsets, xq, wq, torch.float32)
    assert near(out.gu, want, xq, wq, offsets)
    check_y(out.y, out.gu, act)
    low = F.ufp4_gated_gemm(xq, wq, act, offsets=offsets, keep=False)
    assert torch.equal(low.y, out.y.to(torch.bfloat16))


def test_many_groups():
    e, k, f, t = 1024, 32, 3, 1500
    cuts = np.sort(np.random.default_rng(0).integers(0, t + 1, e - 1))
    offsets = torch.from_numpy(np.concatenate([[0], cuts, [t]]).astype(np.int64)).to(DEV)
    xq, wq = quantized(bf(t, k, seed=7)), quantized(bf(e * 2 * f, k, seed=8, std=0.3))
    out = F.ufp4_gated_gemm(xq, wq, F.ACT_SILU, offsets=offsets, out_dtype=torch.float32)
    assert near(out.gu, U.ufp4_grouped_gemm_out(U.FPROP, offsets, xq, wq, torch.float32), xq, wq,
                offsets)


# few output tiles, and enough for the other kernel
@pytest.mark.parametrize("t,f", [(50, 3), (900, 2500)])
def test_odd_offsets(t, f):
    """Offsets that fall, pass the rows or end early: what is in no group stays as
    it was, and nothing beyond the rows is touched."""
    xq, wq = quantized(bf(t, 32, seed=7)), quantized(bf(3 * 2 * f, 32, seed=8, std=0.3))
    for off, mine in (([0, 10, 20, 30], range(30)), ([-5, 10, 5, 9999], range(t)),
                      ([40, 40, 2000, 3000], range(40, t)), ([7, 7, 7, 7], [])):
        y = torch.full((t + 1, f), 7.0, device=DEV)
        gu = torch.full((t + 1, 2 * f), 7.0, device=DEV)
        offsets = torch.tensor(off, device=DEV)
        dx, dw = xq.desc(), wq.desc()
        F._call("ufp4_gated_gemm", y.device, ctypes.byref(dx), ctypes.byref(dw), F.ACT_SILU, 3,
                offsets.data_ptr(), 0, y.data_ptr(), f, gu.data_ptr(), 2 * f)
        left = [i for i in range(t + 1) if i not in set(mine)]
        assert (y[left] == 7.0).all() and (gu[left] == 7.0).all()
        assert (gu[list(mine)] != 7.0).all()


@pytest.mark.parametrize("t,f", [(140, 70), (700, 2501)])
@pytest.mark.parametrize("dtype,code", [(torch.bfloat16, 1), (torch.float32, 0)])
def test_output_strides(t, f, dtype, code):
    """y and gu in rows of any stride; what lies between stays."""
    xq, wq = quantized(bf(t, 64, seed=9)), quantized(bf(2 * f, 64, seed=10, std=0.3))
    ref = F.ufp4_gated_gemm(xq, wq, out_dtype=dtype)
    y = torch.full((t, f + 3), 7.0, dtype=dtype, device=DEV)
    gu = torch.full((t, 2 * f + 5), 7.0, dtype=dtype, device=DEV)
    dx, dw = xq.desc(), wq.desc()
    F._call("ufp4_gated_gemm", y.device, ctypes.byref(dx), ctypes.byref(dw), F.ACT_SILU, 1, None,
            code, y.data_ptr(), f + 3, gu.data_ptr(), 2 * f + 5)
    assert torch.equal(y[:, :f], ref.y) and torch.equal(gu[:, :2 * f], ref.gu)
    assert (y[:, f:] == 7.0).all() and (gu[:, 2 * f:] == 7.0).all()


def test_longest_contraction():
    """65536, one chunk of the GEMM's running sums; a longer one is refused."""
    xq, wq = quantized(bf(5, 65536, seed=11)), quantized(bf(6, 65536, seed=12, std=2.0 ** -8))
    out = F.ufp4_gated_gemm(xq, wq, out_dtype=torch.float32)
    assert near(out.gu, U.ufp4_gemm_out(U.FPROP, xq, wq, torch.float32), xq, wq)
    check_y(out.y, out.gu, F.ACT_SILU)
    xq, wq = quantized(bf(5, 65537, seed=11)), quantized(bf(6, 65537, seed=12))
    with pytest.raises(U.UFP4Error, match="UNSUPPORTED"):
        F.ufp4_gated_gemm(xq, wq)


# -- backward ---------------------------------------------------------------------
def check_bwd(dy, gu, act, got):
    f = dy.shape[1]
    g, u, d = f64(gu[:, :f]), f64(gu[:, f:]), f64(dy)
    value, slope = O.act(g, act)
    ev, es = O.act_error(g, act, EPS32)
    for part, want, err in ((got[:, :f], d * u * slope, np.abs(d * u) * es),
                            (got[:, f:], d * value, np.abs(d) * ev)):
        lim = err + 3 * EPS32 * np.abs(want)
        lim = lim + HALF[dy.dtype] * (np.abs(want) + lim) + TINY
        assert (np.abs(f64(part) - want) <= lim).all()


@pytest.mark.parametrize("rows,f", [(1, 1), (3, 7), (5, 8), (2, 2048), (300, 333), (9, 5000),
                                    (1, 20001), (2000, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ACTS)
def test_backward(rows, f, dtype, act):
    gu, dy = bf(rows, 2 * f, seed=13, std=3.0).to(dtype), bf(rows, f, seed=14, std=1e-2).to(dtype)
    want = F.ufp4_gated_bwd(dy, gu, act)
    check_bwd(dy, gu, act, want)
    # in place, and from rows of other strides and starts
    same = gu.clone()
    before = same._version
    assert torch.equal(F.ufp4_gated_bwd(dy, same, act, out=same), want) and same._version > before
    flat = torch.full((rows * (2 * f + 3) + 1,), float("nan"), dtype=dtype, device=DEV)
    v = flat[1:].view(rows, 2 * f + 3)
    v[:, :2 * f].copy_(gu)
    dv = torch.full((rows, f + 1), float("nan"), dtype=dtype, device=DEV)
    dv[:, :f].copy_(dy)
    assert torch.equal(F.ufp4_gated_bwd(dv[:, :f], v[:, :2 * f], act), want)


@pytest.mark.parametrize("act", ACTS)
def test_backward_over_the_whole_range(act):
    """Gate values from -200 to 200 and at the ends of the type."""
    g = torch.cat([torch.linspace(-200, 200, 4001, device=DEV),
                   torch.linspace(-12, 12, 4001, device=DEV),
                   torch.tensor([-3.0e38, -1e30, -1e-30, -0.0, 0.0, 1e-38, 1e30, 3.0e38],
                                device=DEV)])
    gu = torch.cat([g, torch.ones_like(g)])[None, :]
    dy = torch.ones_like(g)[None, :]
    got = F.ufp4_gated_bwd(dy, gu, act)
    assert got.isfinite().all()
    check_bwd(dy, gu, act, got)


@pytest.mark.parametrize("act", ACTS)
def test_backward_against_differences(act):
    """The forward's own y from FP32 g and u at two nearby points."""
    gu, dy = bf(40, 60, seed=15, std=2.0).float(), bf(40, 30, seed=16).float()
    f, step = 30, 2.0 ** -9
    y = lambda v: O.act(f64(v[:, :f]), act)[0] * f64(v[:, f:])
    got = f64(F.ufp4_gated_bwd(dy, gu, act))
    for j in (0, 7, 29, 30, 59):
        d = torch.zeros_like(gu)
        d[:, j] = step
        diff = ((y(gu + d) - y(gu - d)) / (2 * step) * f64(dy)).sum(1)
        # the third derivatives are below 1 in size: step^2 of |u dy|
        lim = step ** 2 * np.abs(f64(gu)).max() * np.abs(f64(dy)).max() + 1e-4
        assert (np.abs(diff - got[:, j]) <= lim).all(), j


def test_no_rows_and_refusals():
    assert F.ufp4_gated_bwd(torch.empty((0, 4), device=DEV), torch.empty((0, 8), device=DEV)).shape \
        == (0, 8)
    gu, dy = bf(4, 64), bf(4, 32)
    xq, wq = quantized(bf(4, 64)), quantized(bf(6, 64))
    off = torch.tensor([0, 4], device=DEV)
    for call in (lambda: F.ufp4_gated_bwd(dy[:, :31], gu), lambda: F.ufp4_gated_bwd(dy, gu[:, :63]),
                 lambda: F.ufp4_gated_bwd(dy.cpu(), gu), lambda: F.ufp4_gated_bwd(dy, gu, out=dy),
                 lambda: F.ufp4_gated_gemm(xq, quantized(bf(5, 64))),
                 lambda: F.ufp4_gated_gemm(xq, wq, offsets=off.cpu()),
                 lambda: F.ufp4_gated_gemm(xq, wq, offsets=off[:1]),
                 lambda: F.ufp4_gated_gemm(xq, wq, offsets=torch.arange(0, 5, device=DEV))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: F.ufp4_gated_bwd(dy.float(), gu),
                 lambda: F.ufp4_gated_gemm(xq, wq, offsets=off.int()),
                 lambda: F.ufp4_gated_gemm(xq, wq, out_dtype=torch.float64)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: F.ufp4_gated_gemm(xq, wq, F.ACT_NONE), lambda: F.ufp4_gated_bwd(dy, gu, 0),
                 lambda: F.ufp4_gated_gemm(xq, quantized(bf(6, 80))),
                 lambda: F.ufp4_gated_gemm(xq, quantized(bf(6, 64), mask=1))):
        with pytest.raises(U.UFP4Error):
            call()
