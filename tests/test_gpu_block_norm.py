"""RMS norm with residual and E4M3 output, forward and backward, against the
64-bit oracle.

Tolerances (u = 2^-24, an FP32 rounding): a row sum of n terms is at most a
chain of n / 64 additions per lane and 32 more, so it is within
c = (n / 64 + 32) u of the sum of magnitudes; everything computed from it adds
a few u, counted in the 32.  A bf16 result adds half a step, 2^-8; an E4M3
value 2^-4 of itself, or half the smallest step, 2^-10, of its scale."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as O
from uniform_grid_fp4_amd import block as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
EPS = 1e-6
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
TINY = 1e-37                                      # below the normal numbers


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def close(got, want, size, dtype, c, what):
    """|got - want| <= c * size + half a step of the output's type."""
    g = f64(got)
    lim = c * size + HALF[dtype] * (np.abs(want) + c * size) + TINY
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


def inputs(rows, cols, dtype, wtype, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n = lambda s, std: torch.empty(s, device=DEV).normal_(0.0, std, generator=g)
    loud = 1.0 + 30.0 * (torch.rand((cols,), device=DEV, generator=g) < 0.02)
    return ((n((rows, cols), scale) * loud).to(dtype), n((rows, cols), 2.0 * scale).to(dtype),
            (1.0 + n((cols,), 0.2)).to(wtype), n((rows, cols), 1e-2).to(dtype),
            n((rows, cols), 1e-2).to(dtype))


def check_forward(x, w, res, q8=True, out_h=None):
    dtype, (rows, cols) = x.dtype, x.shape
    bf16 = dtype == torch.bfloat16
    h = f64(x) if res is None else O.residual_sum(f64(x), f64(res), bf16)
    y, rstd = O.rmsnorm(h, f64(w), EPS)
    r = B.ufp4_rmsnorm(x, w, res, eps=EPS, q8=q8, out_h=out_h)
    c = (cols / 64 + 32) * U
    assert np.array_equal(f64(r.h), h)
    assert r.y.dtype == dtype and r.rstd.dtype == torch.float32
    assert (np.abs(f64(r.rstd) - rstd) <= c * rstd).all()
    close(r.y, y, np.abs(y), dtype, c, "y")
    if q8:
        scale = np.abs(y).max(1) / O.E4M3_MAX
        s = f64(r.scale)
        assert (np.abs(s - scale) <= 2 * c * scale + TINY).all()
        q = r.q.cpu().to(torch.float32).numpy().astype(np.float64)
        assert (np.abs(q) <= 448).all()
        err = np.abs(q * s[:, None] - y)
        lim = (2.0 ** -4 + 4 * c) * np.abs(y) + s[:, None] * (2.0 ** -10 + 448 * 4 * c) + TINY
        assert (err <= lim).all(), float((err / lim).max())
    return r


SHAPES = [(1, 1), (1, 2048), (3, 7), (2, 8), (5, 63), (4, 64), (3, 65), (7, 511), (2, 1024),
          (33, 1411), (3, 2049), (2, 4104), (2, 6144), (3, 8192), (2, 12289), (2, 16384),
          (1, 40000), (300, 96), (600, 5000), (530, 9000), (3, 11000), (700, 15),
          (1500, 121), (600, 2047), (520, 6143), (600, 1073), (40, 1536)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,wtype", [(torch.bfloat16, torch.bfloat16),
                                         (torch.bfloat16, torch.float32),
                                         (torch.float32, torch.float32)])
def test_forward_and_backward(rows, cols, dtype, wtype):
    x, res, w, dy, dh = inputs(rows, cols, dtype, wtype, rows * 100003 + cols)
    check_forward(x, w, None)
    r = check_forward(x, w, res)
    for d in (None, dh):
        dx, dw = B.ufp4_rmsnorm_bwd(dy, r.h, w, r.rstd, d)
        ex, ew, sx, sw = O.rmsnorm_bwd(f64(dy), f64(r.h), f64(w), EPS,
                                       None if d is None else f64(d))
        c = (cols / 64 + 32) * U
        assert dx.dtype == dtype and dw.dtype == wtype
        close(dx, ex, sx, dtype, 4 * c, "dx")
        close(dw, ew, sw, wtype, (rows + cols / 64 + 32) * U, "dw")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols,ld,start", [(64, 100, 1), (1000, 1003, 3), (2048, 2049, 0),
                                           (6144, 6151, 5), (17, 17, 1)])
def test_strided_and_unaligned_rows(dtype, cols, ld, start):
    """Rows at any stride from any element, NaN around them: same results."""
    x, res, w, dy, dh = inputs(9, cols, dtype, dtype, cols)
    a = check_forward(x, w, res)
    s = [rows_of(t, ld, start) for t in (x, res, dy, dh)]
    b = B.ufp4_rmsnorm(s[0], w, s[1], eps=EPS, q8=True)
    for u, v in zip(a, b):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
    da = B.ufp4_rmsnorm_bwd(dy, a.h, w, a.rstd, dh)
    db = B.ufp4_rmsnorm_bwd(s[2], rows_of(a.h, ld, start), w, a.rstd, s[3])
    assert torch.equal(da[0], db[0]) and torch.equal(da[1], db[1])


def test_residual_stream_in_place():
    for dtype in (torch.bfloat16, torch.float32):
        for which in (0, 1):
            x, res, w, _, _ = inputs(6, 1000, dtype, dtype, 5)
            want = B.ufp4_rmsnorm(x, w, res, q8=True)
            got = B.ufp4_rmsnorm(x, w, res, q8=True, out_h=(x, res)[which])
            assert got.h.data_ptr() == (x, res)[which].data_ptr()
            for u, v in zip(want, got):
                assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


@pytest.mark.parametrize("cols", [5, 127, 1003, 2047, 6143, 9001, 17001])
def test_in_place_where_lanes_share_elements(cols):
    """Rows that end inside a vector, updated in place: the forward's h into x or
    the residual, and (through the C call) dx into dy or dh."""
    for dtype in (torch.bfloat16, torch.float32):
        for which in (0, 1):
            x, res, w, dy, dh = inputs(40, cols, dtype, dtype, cols)
            want = B.ufp4_rmsnorm(x, w, res, q8=True)
            got = B.ufp4_rmsnorm(x, w, res, q8=True, out_h=(x, res)[which])
            for u, v in zip(want, got):
                assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
            dx, dw = B.ufp4_rmsnorm_bwd(dy, want.h, w, want.rstd, dh)
            dw2 = torch.empty_like(dw)
            n = B.ufp4_rmsnorm_bwd_workspace_size(40, cols)
            ws = torch.empty(n, dtype=torch.uint8, device=DEV)
            code = B._CODE[dtype]
            into = (dy, dh)[which]
            st = B.lib().ufp4_rmsnorm_bwd(dy.data_ptr(), cols, want.h.data_ptr(), cols,
                                          w.data_ptr(), want.rstd.data_ptr(), dh.data_ptr(), cols,
                                          code, code, 40, cols, into.data_ptr(), dw2.data_ptr(),
                                          ws.data_ptr(), n, B._stream(torch.device("cuda:0")))
            assert st == 0
            assert torch.equal(into, dx) and torch.equal(dw2, dw)


def test_zero_rows_and_zero_inputs():
    w = torch.ones(96, dtype=torch.bfloat16, device=DEV)
    e = torch.zeros((0, 96), dtype=torch.bfloat16, device=DEV)
    r = B.ufp4_rmsnorm(e, w, e, q8=True)
    assert r.y.shape == (0, 96) and r.scale.shape == (0,)
    dx, dw = B.ufp4_rmsnorm_bwd(e, e, w, r.rstd)
    assert dx.shape == (0, 96) and not dw.any()
    z = torch.zeros((3, 96), dtype=torch.bfloat16, device=DEV)
    r = B.ufp4_rmsnorm(z, w, q8=True)
    assert not r.y.any() and not r.scale.any() and not r.q.float().any()
    assert torch.allclose(r.rstd, torch.full((3,), 1e3, device=DEV))


def test_tiny_rows_keep_their_scale():
    """Rows so small that 448 / max would overflow FP32."""
    x = torch.full((2, 64), 2.0 ** -120, device=DEV)
    x[:, 5] = 2.0 ** -119
    w = torch.full((64,), 2.0 ** -3, device=DEV)
    r = B.ufp4_rmsnorm(x, w, eps=1.0, q8=True)              # rstd 1: y = x / 8
    assert torch.equal(r.q.float()[0, 4:6], torch.tensor([224.0, 448.0], device=DEV))
    assert torch.allclose(r.scale, torch.full((2,), 2.0 ** -122 / 448, device=DEV), rtol=1e-2,
                          atol=0)


def test_nonfinite_rows_stay_in_their_row():
    for bad in (float("inf"), float("nan")):
        for cols in (96, 4096, 20000):
            x, _, w, _, _ = inputs(4, cols, torch.bfloat16, torch.bfloat16, 9)
            want = B.ufp4_rmsnorm(x, w, q8=True)
            x[2, cols // 2] = bad
            got = B.ufp4_rmsnorm(x, w, q8=True)
            keep = [0, 1, 3]
            for u, v in zip(want, got):
                if u is not x and u.data_ptr() != x.data_ptr():
                    assert torch.equal(u[keep].view(torch.uint8), v[keep].view(torch.uint8))
            assert got.q[2].float().isnan().all() and not got.scale[2].isfinite()
            assert not got.y[2, cols // 2].isfinite()


def test_q8_alone_and_custom_workspace():
    x, res, w, dy, _ = inputs(20, 520, torch.bfloat16, torch.bfloat16, 3)
    both = B.ufp4_rmsnorm(x, w, res, q8=True)
    only = B.ufp4_rmsnorm(x, w, res, y=False, q8=True)
    assert only.y is None and torch.equal(only.q.view(torch.uint8), both.q.view(torch.uint8))
    ws = torch.empty(B.ufp4_rmsnorm_bwd_workspace_size(20, 520), dtype=torch.uint8, device=DEV)
    a = B.ufp4_rmsnorm_bwd(dy, both.h, w, both.rstd)
    b = B.ufp4_rmsnorm_bwd(dy, both.h, w, both.rstd, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(Exception):
        B.ufp4_rmsnorm_bwd(dy, both.h, w, both.rstd, workspace=ws[:16])


def test_many_rows_repeat_bit_for_bit():
    x, res, w, dy, dh = inputs(5000, 776, torch.bfloat16, torch.bfloat16, 11)
    r = check_forward(x, w, res)
    a = B.ufp4_rmsnorm_bwd(dy, r.h, w, r.rstd, dh)
    ex, ew, sx, sw = O.rmsnorm_bwd(f64(dy), f64(r.h), f64(w), EPS, f64(dh))
    close(a[0], ex, sx, torch.bfloat16, 4 * (776 / 64 + 32) * U, "dx")
    close(a[1], ew, sw, torch.bfloat16, (5000 + 776 / 64 + 32) * U, "dw")
    for _ in range(3):
        b = B.ufp4_rmsnorm_bwd(dy, r.h, w, r.rstd, dh)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals():
    x, res, w, dy, _ = inputs(4, 64, torch.bfloat16, torch.bfloat16, 1)
    r = B.ufp4_rmsnorm(x, w)
    with pytest.raises(TypeError):
        B.ufp4_rmsnorm(x, w, res.float())
    with pytest.raises(TypeError):
        B.ufp4_rmsnorm(x.float(), w)                        # bf16 weight of float32 rows
    with pytest.raises(ValueError):
        B.ufp4_rmsnorm(x, w, res[:3])
    with pytest.raises(ValueError):
        B.ufp4_rmsnorm(x, w[:63])
    with pytest.raises(ValueError):
        B.ufp4_rmsnorm(x.t(), torch.ones(4, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        B.ufp4_rmsnorm(x, w, out_h=res)
    with pytest.raises(ValueError):
        B.ufp4_rmsnorm(x, w, res.cpu())
    with pytest.raises(ValueError):
        B.ufp4_rmsnorm_bwd(dy, r.h, w, r.rstd[:3])
    with pytest.raises(Exception):
        B.ufp4_rmsnorm(x, w, eps=-1.0)
