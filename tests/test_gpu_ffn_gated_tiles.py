"""The gated product by 128 x 64 tiles, which trains dense layers and experts: its
g and u are bit for bit those of ufp4_gemm_out and ufp4_grouped_gemm_out (the same
blocks added in the same order), are within 1e-5 of the sum of the terms' sizes of
the product in 64 bits of the operands' values, and y is the activation of those
very values.  test_ffn_gated_rule.py holds the sizes to that kernel."""
import ctypes

import numpy as np
import pytest
import torch

from test_gpu_ffn_gated import ACTS, bf, check_y, near, quantized
from uniform_grid_fp4_amd import ffn as F
from uniform_grid_fp4_amd import ufp4 as U

pytestmark = pytest.mark.gpu
DEV = "cuda"
GRIDS = [U.GRID_UNIFORM, U.GRID_E2M1, U.GRID_E2M1_MAX2]

# rows, K, columns: whole tiles; ends within a tile of rows, columns, a stage of K (64)
# and a block of 16; K of one block
DENSE = [(1280, 2048, 1280), (1153, 1000, 1345), (2000, 16, 801), (700, 330, 2501), (4099, 100, 411)]
# rows by expert, K, columns
GROUPED = [([700, 0, 1300, 900], 200, 700), ([129, 1, 0, 640, 127, 128, 0, 300], 2048, 1000),
           ([2900], 96, 601), ([0, 0, 1500, 0], 1000, 1411), ([70] * 64, 72, 1000)]
LONGEST = (1100, 65536, 1450)
# one row's neighbours in the two kernels
SEAM = ((100, 400, 1300), (1500, 400, 1300))
ROWS_OF_A_TILE = 128


def check_whole(y, gu, act):
    """A hundred rows within the activation's bounds, and every row within 64 half
    steps of (1 + |g|) |u|, which covers them."""
    at = torch.unique(torch.linspace(0, len(y) - 1, 100, device=DEV).long())
    check_y(y[at], gu[at], act)
    g, u = gu.double().chunk(2, 1)
    fn = torch.nn.functional.silu if act == F.ACT_SILU else torch.nn.functional.gelu
    assert ((y.double() - fn(g) * u).abs() <= 64 * 2.0 ** -24 * (1 + g.abs()) * u.abs() + 1e-36).all()


def close(gu, xq, wq, offsets=(0,)):
    """Sampled rows against the product in 64 bits."""
    x, w = U.ufp4_dequantize(xq), U.ufp4_dequantize(wq)
    off = [*offsets] if len(offsets) > 1 else [0, xq.rows]
    per = wq.rows // (len(off) - 1)
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        if a == b:
            continue
        at = torch.unique(torch.tensor([a, b - 1, *np.linspace(a, b - 1, 37).astype(int)],
                                       device=DEV))
        xe, we = x[at].double(), w[e * per:(e + 1) * per].double().t().contiguous()
        lim = 1e-5 * (xe.abs() @ we.abs()) + 1e-36
        if not bool(((gu[at].double() - xe @ we).abs() <= lim).all()):
            return False
    return True


@pytest.mark.parametrize("grid", GRIDS)
@pytest.mark.parametrize("t,k,f", DENSE)
def test_dense(t, k, f, grid):
    xq, wq = quantized(bf(t, k, seed=1), grid), quantized(bf(2 * f, k, seed=2, std=2 * k ** -0.5), grid)
    for act in ACTS:
        out = F.ufp4_gated_gemm(xq, wq, act, out_dtype=torch.float32)
        assert torch.equal(out.gu, U.ufp4_gemm_out(U.FPROP, xq, wq, torch.float32))
        check_whole(out.y, out.gu, act)
        low = F.ufp4_gated_gemm(xq, wq, act)
        assert torch.equal(low.gu, out.gu.to(torch.bfloat16))
        assert torch.equal(low.y, out.y.to(torch.bfloat16))
        assert torch.equal(F.ufp4_gated_gemm(xq, wq, act, keep=False).y, low.y)
    assert close(out.gu, xq, wq)


@pytest.mark.parametrize("grid", GRIDS)
@pytest.mark.parametrize("counts,k,f", GROUPED)
def test_grouped(counts, k, f, grid):
    """Each expert's rows with its own weights; empty experts anywhere."""
    e, off = len(counts), np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    offsets = torch.from_numpy(off).to(DEV)
    xq = quantized(bf(int(off[-1]), k, seed=5), grid)
    wq = quantized(bf(e * 2 * f, k, seed=6, std=2 * k ** -0.5), grid)
    want = U.ufp4_grouped_gemm_out(U.FPROP, offsets, xq, wq, torch.float32)
    for act in ACTS:
        out = F.ufp4_gated_gemm(xq, wq, act, offsets=offsets, out_dtype=torch.float32)
        assert torch.equal(out.gu, want)
        check_whole(out.y, out.gu, act)
        low = F.ufp4_gated_gemm(xq, wq, act, offsets=offsets)
        assert torch.equal(low.gu, want.to(torch.bfloat16))
        assert torch.equal(low.y, out.y.to(torch.bfloat16))
        assert torch.equal(F.ufp4_gated_gemm(xq, wq, act, keep=False, offsets=offsets).y, low.y)
    assert close(out.gu, xq, wq, off.tolist())


def test_longest_contraction():
    """65536, one chunk of the running sums."""
    t, k, f = LONGEST
    xq, wq = quantized(bf(t, k, seed=11)), quantized(bf(2 * f, k, seed=12, std=2.0 ** -8))
    out = F.ufp4_gated_gemm(xq, wq, out_dtype=torch.float32)
    assert torch.equal(out.gu, U.ufp4_gemm_out(U.FPROP, xq, wq, torch.float32))
    check_whole(out.y, out.gu, F.ACT_SILU)


@pytest.mark.parametrize("dtype,code", [(torch.bfloat16, 1), (torch.float32, 0)])
def test_strides_and_rows_in_no_group(dtype, code):
    """y and gu in rows of any stride, and offsets that leave rows out: what the
    product has no value for stays as it was."""
    k, f, off = 200, 700, [5, 705, 705, 2005, 2890]
    xq, wq = quantized(bf(2900, k, seed=9)), quantized(bf(4 * 2 * f, k, seed=10, std=0.14))
    offsets = torch.tensor(off, device=DEV)
    y = torch.full((2900, f + 3), 7.0, dtype=dtype, device=DEV)
    gu = torch.full((2900, 2 * f + 5), 7.0, dtype=dtype, device=DEV)
    dx, dw = xq.desc(), wq.desc()
    F._call("ufp4_gated_gemm", y.device, ctypes.byref(dx), ctypes.byref(dw), F.ACT_GELU, 4,
            offsets.data_ptr(), code, y.data_ptr(), f + 3, gu.data_ptr(), 2 * f + 5)
    ref = U.ufp4_grouped_gemm_out(U.FPROP, offsets, xq, wq, torch.float32)
    mine = slice(off[0], off[-1])
    assert torch.equal(gu[mine, :2 * f], ref[mine].to(dtype))
    if dtype == torch.float32:
        check_whole(y[mine, :f], ref[mine], F.ACT_GELU)
    else:
        check_y(y[mine, :f][::29], ref[mine][::29], F.ACT_GELU)
    for t, n in ((y, f), (gu, 2 * f)):
        assert (t[:, n:] == 7.0).all() and (t[:off[0]] == 7.0).all() and (t[off[-1]:] == 7.0).all()


def test_a_row_in_few_tiles_and_in_many():
    """The same row alone and in a batch of the other kernel: the same block terms,
    added up in another order, the same one at every call."""
    (few, k, f), (many, _, _) = SEAM
    xq, wq = quantized(bf(many, k, seed=13)), quantized(bf(2 * f, k, seed=14, std=0.1))
    part = quantized(bf(many, k, seed=13)[:few])
    a = F.ufp4_gated_gemm(part, wq, out_dtype=torch.float32)
    b = F.ufp4_gated_gemm(xq, wq, out_dtype=torch.float32)
    assert near(a.gu, b.gu[:few], part, wq)
    check_whole(a.y, a.gu, F.ACT_SILU)
    assert torch.equal(b.gu, U.ufp4_gemm_out(U.FPROP, xq, wq, torch.float32))
    for q, want in ((part, a), (xq, b)):
        again = F.ufp4_gated_gemm(q, wq, out_dtype=torch.float32)
        assert torch.equal(again.gu, want.gu) and torch.equal(again.y, want.y)
