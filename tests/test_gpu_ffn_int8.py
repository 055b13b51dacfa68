"""Rows in int8 and their product against the oracle: codes, scales and plain
products bit for bit (the sums are exact integers, the FP32 operations after
them the oracle's), gated products within the oracle's bounds of the
activation, its products' roundings (2^-24) and half a step of the type."""
import numpy as np
import pytest
import torch

from oracle import ffn_oracle as O
from uniform_grid_fp4_amd import ffn as F
from uniform_grid_fp4_amd.ufp4 import UFP4Error

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS32 = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: EPS32}
BOTH = [torch.bfloat16, torch.float32]


def values(t):
    return t.detach().cpu().float().numpy()


def normal(rows, cols, dtype=torch.float32, seed=0, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 7919 * rows + cols)
    loud = 1.0 + 20.0 * (torch.rand((cols,), device=DEV, generator=g) < 0.02)
    return (torch.empty((rows, cols), device=DEV).normal_(0.0, std, generator=g) * loud).to(dtype)


def codes(r):
    return r.q[:, :r.k].cpu().numpy().astype(np.int64)


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 3), (2, 7), (5, 64), (4, 127), (4, 128), (4, 129),
                                       (33, 1411), (1, 2048), (600, 96), (3, 6143), (2, 8192),
                                       (2, 20001), (70, 12289), (1000, 16)])
@pytest.mark.parametrize("dtype", BOTH)
def test_codes(rows, cols, dtype):
    x = normal(rows, cols, dtype)
    x[rows // 2] = 0
    r = F.ufp4_int8_quantize(x)
    q, s = O.int8_quantize(values(x))
    assert r.q.shape == (rows, F.int8_kpad(cols)) and r.k == cols
    assert np.array_equal(codes(r), q) and np.array_equal(values(r.scale), s)
    assert not r.q[:, cols:].any()
    flat = torch.full((rows * (cols + 3) + 1,), float("nan"), dtype=dtype, device=DEV)
    v = flat[1:].view(rows, cols + 3)[:, :cols]
    v.copy_(x)
    again = F.ufp4_int8_quantize(v)
    assert torch.equal(again.q, r.q) and torch.equal(again.scale, r.scale)


@pytest.mark.parametrize("cols", [3, 40, 300, 20000])
def test_codes_of_odd_rows(cols):
    """Infinities, NaN, zeros, the smallest and the largest numbers, halves."""
    x = normal(9, cols)
    x[0, cols // 2] = float("inf")
    x[1, 0] = float("nan")
    x[2, cols - 1] = -float("inf")
    x[3] = 0
    x[4] *= 2.0 ** -135
    x[5] = x[5] / x[5].abs().max() * 3.0e38
    x[6] = torch.arange(cols, device=DEV) % 255 - 127.0 + 0.5
    x[6, 0] = 127.0
    x[7] *= 2.0 ** -60
    x[8] = -1.0e-45
    r = F.ufp4_int8_quantize(x)
    q, s = O.int8_quantize(values(x))
    assert np.array_equal(codes(r), q) and np.array_equal(values(r.scale), s, equal_nan=True)
    assert int(r.q.int().abs().max()) <= 127


def operands(m, n, k, seed=0):
    return F.ufp4_int8_quantize(normal(m, k, seed=seed)), \
        F.ufp4_int8_quantize(normal(n, k, seed=seed + 1, std=0.05))


def plain(a, w, bias=None):
    return O.int8_product(codes(a), values(a.scale), codes(w), values(w.scale),
                          None if bias is None else values(bias))


def check_gated(y, p, act):
    f = y.shape[1]
    g, u = p[:, :f].astype(np.float64), p[:, f:].astype(np.float64)
    want = O.act(g, act)[0] * u
    lim = O.act_error(g, act, EPS32)[0] * np.abs(u) + 2 * EPS32 * np.abs(want)
    lim = lim + HALF[y.dtype] * (np.abs(want) + lim) + 1e-36
    assert (np.abs(values(y).astype(np.float64) - want) <= lim).all()


def check(a, w, offsets=None, off=None):
    """All outputs of one pair of operands; `off`: the offsets on the host."""
    n = w.q.shape[0]
    bias = normal(1, n, seed=5)[0].contiguous()
    groups = [(0, a.q.shape[0])] if off is None else list(zip(off[:-1], off[1:]))
    per = n // len(groups)
    rows = [F.Int8Rows(a.q[i:j], a.scale[i:j], a.k) for i, j in groups]
    cols = [F.Int8Rows(w.q[e * per:(e + 1) * per], w.scale[e * per:(e + 1) * per], w.k)
            for e in range(len(groups))]
    for b in (None, bias):
        p = np.concatenate([plain(r, c, None if b is None else b[e * per:(e + 1) * per])
                            for e, (r, c) in enumerate(zip(rows, cols))])
        y = F.ufp4_int8_gemm(a, w, b, offsets=offsets, out_dtype=torch.float32)
        assert np.array_equal(values(y), p)
        y = F.ufp4_int8_gemm(a, w, b, offsets=offsets)
        assert y.dtype == torch.bfloat16 and np.array_equal(values(y), O.round_bf16(p))
        if per % 2 == 0:
            for act in (F.ACT_SILU, F.ACT_GELU):
                y = F.ufp4_int8_gemm(a, w, b, act=act, offsets=offsets, out_dtype=torch.float32)
                assert y.shape == (a.q.shape[0], per // 2)
                check_gated(y, p, act)
                low = F.ufp4_int8_gemm(a, w, b, act=act, offsets=offsets)
                assert torch.equal(low, y.to(torch.bfloat16))


SHAPES = [(1, 1, 1), (1, 2, 7), (1, 34, 128), (2, 64, 129), (15, 16, 200), (16, 18, 640),
          (17, 33, 256), (33, 100, 300), (64, 30, 64), (65, 66, 100), (127, 130, 129),
          (128, 128, 128), (129, 300, 257), (300, 257, 1411), (257, 512, 512)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_products(m, n, k):
    check(*operands(m, n, k))


@pytest.mark.parametrize("m,n", [(1, 2048), (700, 16384), (2111, 4100)])
def test_large_tiles(m, n):
    """Enough output for the largest tiles; sampled rows against the oracle."""
    a, w = operands(m, n, 384, seed=3)
    pick = torch.tensor(sorted({0, m // 3, m // 2, m - 1}), device=DEV)
    p = plain(F.Int8Rows(a.q[pick], a.scale[pick], a.k), w)
    y = F.ufp4_int8_gemm(a, w, out_dtype=torch.float32)
    assert np.array_equal(values(y[pick]), p)
    g = F.ufp4_int8_gemm(a, w, act=F.ACT_SILU, out_dtype=torch.float32)
    check_gated(g[pick], p, F.ACT_SILU)
    # the same rows by themselves: another kernel, the same bits
    few = F.Int8Rows(a.q[pick], a.scale[pick], a.k)
    assert torch.equal(F.ufp4_int8_gemm(few, w, out_dtype=torch.float32), y[pick])
    assert torch.equal(F.ufp4_int8_gemm(few, w, act=F.ACT_SILU, out_dtype=torch.float32), g[pick])


@pytest.mark.parametrize("counts", [[8100], [3000, 0, 1, 5000, 700]])
def test_large_tiles_of_several_rounds(counts):
    """Workgroups that go on to other tiles: every row against the same rows in calls
    of their own, which take other tiles, and some against the oracle."""
    m, e, n, k = sum(counts), len(counts), 8192, 1411
    off = [0, *torch.tensor(counts).cumsum(0).tolist()]
    a, w = operands(m, e * n, k, seed=7)
    offsets = torch.tensor(off, device=DEV) if e > 1 else None
    for act, dtype in ((F.ACT_NONE, torch.float32), (F.ACT_NONE, torch.bfloat16),
                       (F.ACT_SILU, torch.float32), (F.ACT_GELU, torch.bfloat16)):
        y = F.ufp4_int8_gemm(a, w, act=act, offsets=offsets, out_dtype=dtype)
        for g in range(e):
            mine = F.Int8Rows(w.q[g * n:(g + 1) * n], w.scale[g * n:(g + 1) * n], k)
            for r in range(off[g], off[g + 1], 400):
                to = min(r + 400, off[g + 1])
                few = F.ufp4_int8_gemm(F.Int8Rows(a.q[r:to], a.scale[r:to], k), mine, act=act,
                                       out_dtype=dtype)
                assert torch.equal(y[r:to], few), (act, dtype, g, r)
        if act == F.ACT_NONE and dtype == torch.float32:
            at = off[1] - 1
            p = plain(F.Int8Rows(a.q[at:at + 1], a.scale[at:at + 1], k),
                      F.Int8Rows(w.q[:n], w.scale[:n], k))
            assert np.array_equal(values(y[at:at + 1]), p)


@pytest.mark.parametrize("m,n,k", [(65, 66, 513), (129, 300, 900), (1000, 70, 6080), (70, 34, 131),
                                   (905, 1536, 1411), (460, 2050, 1300)])
def test_few_tiles_of_a_long_contraction(m, n, k):
    """Tiles that split K over their waves, with a number of stages that the parts
    share and with one that they do not."""
    check(*operands(m, n, k))


@pytest.mark.parametrize("counts", [[65, 0, 66, 64, 1, 70], [300, 20, 140]])
def test_grouped_few_tiles(counts):
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    for n, k in ((34, 1411), (258, 640)):
        a, w = operands(int(off[-1]), n * len(counts), k)
        check(a, w, torch.from_numpy(off).to(DEV), off)


COUNTS = [[5, 0, 130, 1, 0, 64], [0, 0, 7], [40], [1] * 70, [0, 129], [300, 0, 280, 3],
          [0, 0], [0, 33, 0, 0, 0, 0, 0, 0]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("n,k", [(34, 100), (130, 256)])
def test_grouped(counts, n, k):
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    a, w = operands(int(off[-1]), n * len(counts), k)
    check(a, w, torch.from_numpy(off).to(DEV), off)


def test_many_groups_and_odd_offsets():
    """1024 experts; then offsets that fall, pass the rows or end early, with
    both kernels: what is in no group stays as it was."""
    import ctypes
    rng = np.random.default_rng(0)
    for t in (900, 90000):
        off = np.concatenate([[0], np.sort(rng.integers(0, t + 1, 1023)), [t]]).astype(np.int64)
        a, w = operands(t, 1024 * 4, 64)
        offsets = torch.from_numpy(off).to(DEV)
        y = F.ufp4_int8_gemm(a, w, offsets=offsets, out_dtype=torch.float32)
        expert = np.searchsorted(off[1:], np.arange(t), side="right")
        for i in rng.integers(0, t, 60):
            e = expert[i]
            p = plain(F.Int8Rows(a.q[i:i + 1], a.scale[i:i + 1], 64),
                      F.Int8Rows(w.q[4 * e:4 * e + 4], w.scale[4 * e:4 * e + 4], 64))
            assert np.array_equal(values(y[i:i + 1]), p)
    for t in (50, 500):
        a, w = operands(t, 3 * 6, 64)
        for off, mine in (([0, 10, 20, 30], range(30)), ([-5, 10, 5, 9999], range(t)),
                          ([40, 40, 20000, 30000], range(40, t)), ([7, 7, 7, 7], [])):
            y = torch.full((t + 1, 6), 7.0, device=DEV)
            offsets = torch.tensor(off, device=DEV)
            da, dw = F._int8_operand(a, "a", y.device), F._int8_operand(w, "w", y.device)
            F._call("ufp4_int8_gemm", y.device, da.buffer_info()[0], dw.buffer_info()[0], None,
                    F.ACT_NONE, 3, offsets.data_ptr(), 0, y.data_ptr(), 6)
            left = [i for i in range(t + 1) if i not in set(mine)]
            assert (y[left] == 7.0).all() and (y[list(mine)] != 7.0).all()
        assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_extremes():
    """The longest contraction at the largest codes (-128 among them, which the
    quantizer never makes): sums up to 2^31 - 2^14; longer is refused."""
    k = 131071
    for m in (2, 70):
        q = torch.zeros((m, F.int8_kpad(k)), dtype=torch.int8, device=DEV)
        q[:, :k] = -128
        q[1, :k] = 127
        a = F.Int8Rows(q, torch.ones(m, device=DEV), k)
        y = F.ufp4_int8_gemm(a, a, out_dtype=torch.float32)
        want = np.array([[128 * 128 * k, -128 * 127 * k], [-128 * 127 * k, 127 * 127 * k]], np.int64)
        assert np.array_equal(values(y[:2, :2]), want.astype(np.float32))
    big = F.Int8Rows(torch.zeros((1, 131072), dtype=torch.int8, device=DEV),
                     torch.ones(1, device=DEV), 131072)
    with pytest.raises(UFP4Error, match="UNSUPPORTED"):
        F.ufp4_int8_gemm(big, big)
    # what one operand holds past k does not matter where the other has zeros
    a, w = operands(40, 30, 100)
    y = F.ufp4_int8_gemm(a, w)
    w.q[:, 100:] = 77
    assert torch.equal(F.ufp4_int8_gemm(a, w), y)


def test_scales_that_are_not_finite_stay_in_their_rows():
    x = normal(70, 100)
    x[3, 5], x[66, 0] = float("nan"), float("inf")
    w = F.ufp4_int8_quantize(normal(20, 100, seed=2))
    for act, n in ((F.ACT_NONE, 20), (F.ACT_SILU, 10)):
        for part in (x, x[:10]):
            y = F.ufp4_int8_linear(part, w, act=act)
            bad = {3, 66} & set(range(part.shape[0]))
            for i in range(part.shape[0]):
                assert bool(y[i].isnan().all()) == (i in bad) and y.shape[1] == n
                assert bool(y[i].isfinite().all()) == (i not in bad)


@pytest.mark.parametrize("m", [1, 20, 300])
@pytest.mark.parametrize("dtype", BOTH)
def test_linear_is_quantize_then_product(m, dtype):
    x = normal(m, 130, dtype)
    w = F.ufp4_int8_quantize(normal(48, 130, seed=2))
    bias = normal(1, 48, seed=3)[0].contiguous()
    offsets = torch.tensor([0, m // 2, m, m], device=DEV)
    for kw in (dict(), dict(bias=bias), dict(act=F.ACT_GELU), dict(offsets=offsets),
               dict(offsets=offsets, act=F.ACT_SILU, bias=bias)):
        y = F.ufp4_int8_linear(x, w, **kw)
        assert y.dtype == dtype
        want = F.ufp4_int8_gemm(F.ufp4_int8_quantize(x), w, out_dtype=dtype, **kw)
        assert torch.equal(y, want)
        flat = torch.full((m, 150), float("nan"), dtype=dtype, device=DEV)
        flat[:, 3:133].copy_(x)
        ws = torch.empty(F.ufp4_int8_linear_workspace_size(m, 130, True), dtype=torch.uint8, device=DEV)
        assert torch.equal(F.ufp4_int8_linear(flat[:, 3:133], w, workspace=ws, **kw), y)


@pytest.mark.parametrize("m,k", [(1, 1), (1, 7), (1, 130), (1, 2048), (1, 32768), (1, 32641),
                                 (2, 5000), (2, 8192), (3, 5000), (3, 10000), (4, 4096), (4, 8192),
                                 (5, 100), (7, 2200), (7, 4000), (8, 2048), (8, 4096), (9, 1700),
                                 (9, 3500), (15, 1000), (15, 2000), (16, 1024), (16, 2048),
                                 (16, 130), (16, 3)])
@pytest.mark.parametrize("dtype", BOTH)
def test_few_rows_quantized_by_the_product(m, k, dtype):
    """Bit for bit what the two calls give, at the rows' ends, zero rows and rows
    that are not finite among them."""
    fuses = F.ufp4_int8_linear_workspace_size(m, k) == 0
    assert fuses == (m == 1 or m * F.int8_kpad(k) <= 16384)
    x, w = normal(m, k, dtype), F.ufp4_int8_quantize(normal(38, k, seed=2, std=0.05))
    bias = normal(1, 38, seed=3)[0].contiguous()
    for i in range(3):
        for kw in (dict(), dict(bias=bias), dict(act=F.ACT_SILU), dict(act=F.ACT_GELU, bias=bias)):
            want = F.ufp4_int8_gemm(F.ufp4_int8_quantize(x), w, out_dtype=dtype, **kw)
            y = F.ufp4_int8_linear(x, w, **kw)
            assert torch.equal(y.nan_to_num(7.0), want.nan_to_num(7.0)), (i, kw)
        x = x.clone()
        if i == 0:
            x[m // 2] = 0
        else:
            x[m - 1, k - 1] = float("nan")
    flat = torch.full((m, k + 5), float("nan"), dtype=dtype, device=DEV)
    x = normal(m, k, dtype)
    flat[:, 3:3 + k].copy_(x)
    assert torch.equal(F.ufp4_int8_linear(flat[:, 3:3 + k], w), F.ufp4_int8_linear(x, w))


def test_output_rows_of_any_stride():
    a, w = operands(70, 40, 64)
    for m in (9, 70):
        part = F.Int8Rows(a.q[:m], a.scale[:m], 64)
        want = F.ufp4_int8_gemm(part, w)
        y = torch.full((m, 43), 7.0, dtype=torch.bfloat16, device=DEV)
        da, dw = F._int8_operand(part, "a", y.device), F._int8_operand(w, "w", y.device)
        F._call("ufp4_int8_gemm", y.device, da.buffer_info()[0], dw.buffer_info()[0], None,
                F.ACT_NONE, 1, None, 1, y.data_ptr(), 43)
        assert torch.equal(y[:, :40], want) and (y[:, 40:] == 7.0).all()


def test_no_rows_and_refusals():
    w = F.ufp4_int8_quantize(normal(6, 64))
    none = torch.empty((0, 64), device=DEV)
    assert F.ufp4_int8_quantize(none).q.shape == (0, 128)
    assert F.ufp4_int8_linear(none, w).shape == (0, 6)
    assert F.ufp4_int8_linear(none, w, act=F.ACT_SILU).shape == (0, 3)
    a = F.ufp4_int8_quantize(normal(4, 64))
    x = normal(4, 64)
    off = torch.tensor([0, 2, 4], device=DEV)
    bad_q = F.Int8Rows(a.q[:, ::2], a.scale, 64)
    for call in (lambda: F.ufp4_int8_gemm(a, F.ufp4_int8_quantize(normal(6, 65))),
                 lambda: F.ufp4_int8_linear(x[:, :63], w), lambda: F.ufp4_int8_gemm(bad_q, w),
                 lambda: F.ufp4_int8_gemm(F.Int8Rows(a.q, a.scale[:3], 64), w),
                 lambda: F.ufp4_int8_gemm(F.Int8Rows(a.q, a.scale, 200), w),
                 lambda: F.ufp4_int8_gemm(a, F.Int8Rows(w.q[:5], w.scale[:5], 64), act=F.ACT_SILU),
                 lambda: F.ufp4_int8_gemm(a, F.Int8Rows(w.q[:5], w.scale[:5], 64), offsets=off),
                 lambda: F.ufp4_int8_gemm(a, w, bias=torch.zeros(5, device=DEV)),
                 lambda: F.ufp4_int8_gemm(a, w, offsets=off.cpu()),
                 lambda: F.ufp4_int8_gemm(a, F.Int8Rows(w.q[:0], w.scale[:0], 64)),
                 lambda: F.ufp4_int8_gemm(a, F.Int8Rows(w.q.cpu(), w.scale, 64)),
                 lambda: F.ufp4_int8_quantize(x.t())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: F.ufp4_int8_gemm(a, w, out_dtype=torch.float16),
                 lambda: F.ufp4_int8_gemm(a, w, bias=torch.zeros(6, device=DEV).bfloat16()),
                 lambda: F.ufp4_int8_gemm(a, w, offsets=off.int()),
                 lambda: F.ufp4_int8_gemm(F.Int8Rows(a.q.view(torch.uint8), a.scale, 64), w)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(UFP4Error):
        F.ufp4_int8_gemm(a, w, act=7)
    with pytest.raises(UFP4Error):
        F.ufp4_int8_linear(normal(40, 64), w, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
