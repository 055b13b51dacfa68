"""Layer norm with residual, forward and backward, against the 64-bit oracle.

Tolerances (u = 2^-24, an FP32 rounding): a row sum of n terms is at most a
chain of n / 64 additions per lane and 32 more, so it is within c = (n / 64 +
32) u of the sum of magnitudes.  The mean is off by at most dev = c mean|h|.  A
shift of the centre by dev changes the variance by dev^2, the sums by c of
itself, so rstd is off by rel = c + dev^2 / (2 (var + eps)) and a few u, counted
in the c's 32.  From there on every term carries rel and c, and the shift
itself: rstd dev.  A bf16 result adds half a step, 2^-8."""
import numpy as np
import pytest
import torch

from oracle import ffn_oracle as O
from uniform_grid_fp4_amd import ffn as F

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
EPS = 1e-5
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
TINY = 1e-37                                      # below the normal numbers
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
         (torch.float32, torch.float32)]


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def close(got, want, lim, dtype, what):
    """|got - want| <= lim + half a step of the output's type."""
    g = f64(got)
    lim = lim + HALF[dtype] * (np.abs(want) + lim) + TINY
    bad = ~(np.abs(g - want) <= lim)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, worst ratio "
                           f"{np.nanmax(np.abs(g - want) / lim):.3g}")


def rows_of(t, ld, start=0):
    """t's values in rows of stride ld that begin `start` elements in."""
    n, h = t.shape
    flat = torch.full((start + n * ld + 3,), float("nan"), dtype=t.dtype, device=DEV)
    v = flat[start:start + n * ld].view(n, ld)[:, :h]
    v.copy_(t)
    return v


def inputs(rows, cols, dtype, wtype, seed, shift=0.5):
    """x, residual, weight, bias, dy, dh; the rows have means of their own."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n = lambda s, std: torch.empty(s, device=DEV).normal_(0.0, std, generator=g)
    loud = 1.0 + 30.0 * (torch.rand((cols,), device=DEV, generator=g) < 0.02)
    return ((n((rows, cols), 1.0) * loud + n((rows, 1), shift)).to(dtype),
            n((rows, cols), 2.0).to(dtype), (1.0 + n((cols,), 0.2)).to(wtype),
            n((cols,), 0.3).to(wtype), n((rows, cols), 1e-2).to(dtype),
            n((rows, cols), 1e-2).to(dtype))


def errors(h, eps=EPS):
    """(c, dev, rel) of rows h."""
    c = (h.shape[1] / 64 + 32) * U
    dev = c * np.abs(h).mean(1)
    return c, dev, c + dev ** 2 / (2 * (h.var(1) + eps) + 1e-300)


def check_forward(x, w, b, res, out_h=None, eps=EPS):
    dtype = x.dtype
    h = f64(x) if res is None else O.residual_sum(f64(x), f64(res), dtype == torch.bfloat16)
    y, mean, rstd, xhat = O.layernorm(h, f64(w), None if b is None else f64(b), eps)
    r = F.ufp4_layernorm(x, w, b, res, eps=eps, out_h=out_h)
    c, dev, rel = errors(h, eps)
    assert np.array_equal(f64(r.h), h)
    assert r.y.dtype == dtype and r.rstd.dtype == r.mean.dtype == torch.float32
    assert (np.abs(f64(r.mean) - mean) <= dev + TINY).all()
    assert (np.abs(f64(r.rstd) - rstd) <= rel * rstd).all()
    aw = np.abs(f64(w))
    lim = (rstd * dev)[:, None] * aw + (rel + 4 * U)[:, None] * np.abs(xhat * f64(w)) \
        + 2 * U * np.abs(y)
    close(r.y, y, lim, dtype, "y")
    return r


def check_backward(dy, r, w, b, dh, eps=EPS):
    rows, cols = dy.shape
    h, gy, gw = f64(r.h), f64(dy), f64(w)
    dx, dw, db = F.ufp4_layernorm_bwd(dy, r.h, w, r.mean, r.rstd, dh, bias=b is not None)
    d = 0.0 if dh is None else f64(dh)
    ex, ew, eb = O.layernorm_bwd(gy, h, gw, eps, d)
    _, _, rstd, xhat = O.layernorm(h, gw, None, eps)
    c, dev, rel = errors(h, eps)
    off = (rstd * dev)[:, None] + (rel + 4 * U)[:, None] * np.abs(xhat)      # of xhat
    g = np.abs(gy * gw)
    inner = (g * np.abs(xhat)).mean(1, keepdims=True)
    size = g + g.mean(1, keepdims=True) + np.abs(xhat) * inner
    lim = rstd[:, None] * ((rel[:, None] + 4 * c) * size + off * inner
                           + np.abs(xhat) * (g * off).mean(1, keepdims=True)) + 2 * U * np.abs(d)
    assert dx.dtype == dy.dtype and dw.dtype == w.dtype
    close(dx, ex, lim, dy.dtype, "dx")
    long = (rows + 96) * U                           # the chain over the rows, and the slices
    close(dw, ew, (np.abs(gy) * (long * np.abs(xhat) + off)).sum(0), w.dtype, "dw")
    if b is None:
        assert db is None
    else:
        close(db, eb, long * np.abs(gy).sum(0), w.dtype, "db")
    return dx, dw, db


SHAPES = [(1, 1), (1, 2048), (3, 7), (2, 8), (5, 63), (4, 64), (3, 65), (7, 511), (2, 1024),
          (33, 1411), (3, 2049), (2, 4104), (2, 6144), (3, 8192), (2, 12289), (2, 16384),
          (1, 40000), (300, 96), (600, 5000), (530, 9000), (3, 11000), (700, 15),
          (1500, 121), (600, 2047), (520, 6143), (600, 1073), (40, 1536), (1500, 2000),
          (1300, 1601), (600, 8000), (300, 15001), (270, 16000), (2300, 1300), (4500, 512),
          (20000, 100)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,wtype", TYPES)
def test_forward_and_backward(rows, cols, dtype, wtype):
    x, res, w, b, dy, dh = inputs(rows, cols, dtype, wtype, rows * 100003 + cols)
    check_forward(x, w, None, None)
    r = check_forward(x, w, b, res)
    check_backward(dy, r, w, b, None)
    check_backward(dy, r, w, None, dh)


@pytest.mark.parametrize("cols", [5, 300, 2048, 20000])
def test_far_from_zero(cols):
    """Rows whose mean is 4000 times their spread: the squares are those of
    the centred values."""
    x, _, w, b, dy, _ = inputs(6, cols, torch.float32, torch.float32, cols, shift=0.0)
    r = check_forward(x + 4000.0, w, b, None)
    check_backward(dy, r, w, b, None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols,ld,start", [(64, 100, 1), (1000, 1003, 3), (2048, 2049, 0),
                                           (6144, 6151, 5), (17, 17, 1), (20000, 20007, 1)])
def test_strided_and_unaligned_rows(dtype, cols, ld, start):
    """Rows at any stride from any element, NaN around them: same results."""
    x, res, w, b, dy, dh = inputs(9, cols, dtype, dtype, cols)
    a = check_forward(x, w, b, res)
    s = [rows_of(t, ld, start) for t in (x, res, dy, dh)]
    r = F.ufp4_layernorm(s[0], w, b, s[1], eps=EPS)
    assert all(torch.equal(p, q) for p, q in zip(a, r))
    want = F.ufp4_layernorm_bwd(dy, a.h, w, a.mean, a.rstd, dh)
    hs = rows_of(a.h, ld, start)
    got = F.ufp4_layernorm_bwd(s[2], hs, w, a.mean, a.rstd, s[3])
    assert all(torch.equal(p, q) for p, q in zip(want, got))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [64, 121, 2047, 2048, 6143, 20001])
def test_in_place(dtype, cols):
    """The stream updated in place, and dx over dy or dh, also where two lanes
    share elements."""
    x, res, w, b, dy, dh = inputs(70, cols, dtype, dtype, cols + 1)
    want = F.ufp4_layernorm(x, w, b, res, eps=EPS)
    for into in (0, 1):
        pair = [x.clone(), res.clone()]
        version = pair[into]._version
        got = F.ufp4_layernorm(pair[0], w, b, pair[1], eps=EPS, out_h=pair[into])
        assert got.h.data_ptr() == pair[into].data_ptr() and pair[into]._version > version
        assert all(torch.equal(p, q) for p, q in zip(want, got))
    gx, gw, gb = F.ufp4_layernorm_bwd(dy, want.h, w, want.mean, want.rstd, dh)
    ws = torch.empty(F.ufp4_layernorm_bwd_workspace_size(70, cols), dtype=torch.uint8, device=DEV)
    for into in (0, 1):
        pair = [dy.clone(), dh.clone()]
        dw, db = torch.empty_like(w), torch.empty_like(w)
        code = 1 if dtype == torch.bfloat16 else 0
        F._call("ufp4_layernorm_bwd", x.device, pair[0].data_ptr(), cols, want.h.data_ptr(), cols,
                w.data_ptr(), want.mean.data_ptr(), want.rstd.data_ptr(), pair[1].data_ptr(), cols,
                code, code, 70, cols, pair[into].data_ptr(), dw.data_ptr(), db.data_ptr(),
                ws.data_ptr(), ws.numel())
        assert torch.equal(pair[into], gx) and torch.equal(dw, gw) and torch.equal(db, gb)


def test_rows_that_are_not_finite_stay_alone():
    x, res, w, b, dy, _ = inputs(6, 300, torch.float32, torch.float32, 5)
    x[1, 7], x[3, 299], x[4, 0] = float("nan"), float("inf"), -float("inf")
    r = F.ufp4_layernorm(x, w, b, eps=EPS)
    for i in range(6):
        assert bool(r.y[i].isnan().all()) == (i in (1, 3, 4))
        assert bool(r.y[i].isfinite().all()) == (i not in (1, 3, 4))
    dx, dw, db = F.ufp4_layernorm_bwd(dy, r.h, w, r.mean, r.rstd)
    assert dw.isnan().all() and db.isfinite().all()
    assert dx[[0, 2, 5]].isfinite().all() and dx[[1, 3, 4]].isnan().all()


@pytest.mark.parametrize("cols", [1, 3, 64, 300, 2048, 9000, 20000])
def test_constant_rows(cols):
    """No spread at all: y is the bias, and the gradient of the row is what is
    left of g's mean; large constants overflow nothing outside the row."""
    w, b = torch.full((cols,), 2.0, device=DEV), torch.full((cols,), 0.25, device=DEV)
    for value in (0.0, 1.0, -1024.0, 2.0 ** 100):
        x = torch.full((3, cols), value, device=DEV)
        r = F.ufp4_layernorm(x, w, b, eps=EPS)
        # a power of two sums exactly while the partial sums are below 2^24 of it
        assert torch.equal(r.y, torch.full_like(x, 0.25)) and torch.equal(r.mean, x[:, 0])
        dy = torch.ones_like(x)
        dx, dw, db = F.ufp4_layernorm_bwd(dy, r.h, w, r.mean, r.rstd)
        assert not dx.any() and not dw.any() and torch.equal(db, torch.full_like(w, 3.0))


def test_no_rows():
    x, w = torch.empty((0, 64), device=DEV), torch.ones(64, device=DEV)
    r = F.ufp4_layernorm(x, w, w, x)
    assert r.y.shape == (0, 64) and r.mean.shape == (0,)
    dx, dw, db = F.ufp4_layernorm_bwd(x, x, w, r.mean, r.rstd)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_gradient_against_differences():
    """The kernels' own forward pass, moved along a random direction, in FP32:
    L = <y, dy> + <h, dh> changes by <dx, d>.  The forward's values are good to
    about 2^-22 of L's terms, and the step divides that."""
    x, res, w, b, dy, dh = inputs(4, 200, torch.float32, torch.float32, 77)
    step = 2.0 ** -7
    dx = None
    for what in range(3):
        d = torch.randn((x, w, b)[what].shape, device=DEV)

        def value(t):
            a = [x, w, b]
            a[what] = a[what] + t * d
            r = F.ufp4_layernorm(a[0], a[1], a[2], res, eps=EPS)
            return float((r.y.double() * dy.double()).sum() + (r.h.double() * dh.double()).sum()), r

        (up, _), (down, _), (_, r) = value(step), value(-step), value(0.0)
        grads = F.ufp4_layernorm_bwd(dy, r.h, w, r.mean, r.rstd, dh)
        want = float((grads[what].double() * d.double()).sum())
        size = float((r.y.abs().double() * dy.abs().double()).sum()
                     + (r.h.abs().double() * dh.abs().double()).sum())
        # the third derivative's part: step^2 / 6 of a slope of 4 such sizes
        lim = 2.0 ** -20 * size / step + step ** 2 * size
        assert abs((up - down) / (2 * step) - want) <= lim, (what, up, down, want, lim)


def test_refusals():
    x, res, w, b, dy, _ = inputs(4, 64, torch.bfloat16, torch.bfloat16, 1)
    r = F.ufp4_layernorm(x, w, b)
    for call in (lambda: F.ufp4_layernorm(x, w[:32], b), lambda: F.ufp4_layernorm(x, w, b[:32]),
                 lambda: F.ufp4_layernorm(x, w, b, res[:3]), lambda: F.ufp4_layernorm(x[0], w),
                 lambda: F.ufp4_layernorm(x.t(), w[:4]), lambda: F.ufp4_layernorm(x, w, out_h=x),
                 lambda: F.ufp4_layernorm(x, w, b, res, out_h=x[:, :32]),
                 lambda: F.ufp4_layernorm_bwd(dy, r.h, w, r.mean[:3], r.rstd),
                 lambda: F.ufp4_layernorm_bwd(dy, r.h, w, r.mean, r.rstd.cpu()),
                 lambda: F.ufp4_layernorm_bwd(dy[:, :32], r.h, w, r.mean, r.rstd),
                 lambda: F.ufp4_layernorm(x, w.cpu())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: F.ufp4_layernorm(x, w, b.float()), lambda: F.ufp4_layernorm(x.float(), w),
                 lambda: F.ufp4_layernorm(x, w, b, res.float()),
                 lambda: F.ufp4_layernorm_bwd(dy.float(), r.h, w, r.mean, r.rstd),
                 lambda: F.ufp4_layernorm_bwd(dy, r.h, w, r.mean.double(), r.rstd)):
        with pytest.raises(TypeError):
            call()
    from uniform_grid_fp4_amd.ufp4 import UFP4Error
    with pytest.raises(UFP4Error):
        F.ufp4_layernorm(x, w, b, eps=-1.0)
    with pytest.raises(UFP4Error):
        F.ufp4_layernorm_bwd(dy, r.h, w, r.mean, r.rstd,
                             workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
