"""The feed-forward operators' C ABI without a GPU: every function that
include/ufp4_ffn.h declares is exported, bad arguments are refused on the host
before anything is enqueued, and the binding refuses tensors of wrong types,
shapes, strides or devices."""
import contextlib
import ctypes
import os
import re
import types

import pytest
import torch

from uniform_grid_fp4_amd import block as B
from uniform_grid_fp4_amd import ffn as F
from uniform_grid_fp4_amd import ufp4 as U

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16 = U.OUT_F32, U.OUT_BF16
A = 0x10000                # an address that is never dereferenced
BIG = 1 << 40


class Rows(ctypes.Structure):
    """Mirror of ufp4_int8_rows."""
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("k", ctypes.c_int64)]


def test_library_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "ufp4_ffn.h")).read()
    decl = sorted(set(re.findall(r"^(?:ufp4_status|size_t)\s+(ufp4_\w+)\(", src, re.M)))
    assert sorted(F.EXPORTS) == decl
    for name in decl:
        assert hasattr(F.lib(), name), name


def norm(**kw):
    a = dict(x=A, ld=64, res=A, ldr=64, w=A, b=A, dt=BF16, wdt=BF16, rows=4, cols=64, eps=1e-6,
             h=A, y=A, mean=A, rstd=A)
    a.update(kw)
    return F.lib().ufp4_layernorm(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(h=None), -1), (dict(rstd=None), -1),
    (dict(mean=None), -1), (dict(y=None), -1), (dict(x=A + 1), -1), (dict(res=A + 1), -1),
    (dict(h=A + 1), -1), (dict(y=A + 1), -1), (dict(w=A + 1), -1), (dict(b=A + 1), -1),
    (dict(mean=A + 2), -1), (dict(rstd=A + 2), -1), (dict(dt=2), -1), (dict(wdt=3), -1),
    (dict(dt=F32, wdt=BF16), -1), (dict(dt=F32, wdt=F32, x=A + 2), -1),
    (dict(wdt=F32, b=A + 2), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(rows=-1), -2), (dict(cols=0), -2), (dict(ld=63), -2), (dict(ldr=63), -2),
    (dict(cols=(1 << 24) + 1, ld=BIG, ldr=BIG), -2), (dict(rows=(1 << 40) + 1), -2),
    (dict(rows=1 << 40, cols=1 << 24, ld=BIG, ldr=BIG), -2),   # the product passes 63 bits
    (dict(rows=1 << 30, ld=1 << 31), -2),                      # the last row past 2^60
    (dict(rows=0, x=None, h=None, y=None, mean=None, rstd=None), 0),    # nothing to do
])
def test_layernorm_rejects(kw, expect):
    assert norm(**kw) == expect


def norm_bwd(**kw):
    a = dict(dy=A, ldy=64, h=A, ldh=64, w=A, mean=A, rstd=A, dh=A, ldd=64, dt=BF16, wdt=BF16,
             rows=4, cols=64, dx=A, dw=A, db=A, ws=A, n=1 << 20)
    a.update(kw)
    return F.lib().ufp4_layernorm_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dy=None), -1), (dict(h=None), -1), (dict(w=None), -1), (dict(mean=None), -1),
    (dict(rstd=None), -1), (dict(dx=None), -1), (dict(dw=None), -1), (dict(ws=None), -1),
    (dict(n=0), -1), (dict(n=2 * 64 * 4 - 1), -1), (dict(ws=A + 8), -1), (dict(dy=A + 1), -1),
    (dict(dh=A + 1), -1), (dict(dx=A + 1), -1), (dict(dw=A + 1), -1), (dict(db=A + 1), -1),
    (dict(dt=7), -1), (dict(dt=F32, wdt=BF16), -1), (dict(ldy=3), -2), (dict(ldh=3), -2),
    (dict(ldd=3), -2), (dict(cols=-1), -2), (dict(rows=-2), -2),
    (dict(rows=1 << 40, cols=1 << 24, ldy=BIG, ldh=BIG, ldd=BIG), -2),
])
def test_layernorm_bwd_rejects(kw, expect):
    assert norm_bwd(**kw) == expect


def dropout(**kw):
    a = dict(x=A, ld=64, res=A, ldr=64, dt=BF16, rows=4, cols=64, p=0.1, seed=1, off=0, doff=None,
             y=A)
    a.update(kw)
    return F.lib().ufp4_dropout(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), -1), (dict(y=None), -1), (dict(x=A + 1), -1), (dict(res=A + 1), -1),
    (dict(y=A + 1), -1), (dict(dt=F32, y=A + 2), -1), (dict(doff=A + 4), -1), (dict(dt=2), -1),
    (dict(p=-0.01), -1), (dict(p=1.01), -1), (dict(p=float("nan")), -1), (dict(rows=-1), -2),
    (dict(cols=0), -2), (dict(ld=63), -2), (dict(ldr=63), -2), (dict(rows=(1 << 40) + 1), -2),
    (dict(rows=0, x=None, y=None), 0),
])
def test_dropout_rejects(kw, expect):
    assert dropout(**kw) == expect


def operand(rows, k=64, grid=0, rht=0, mask=0, codes=A, scales=A, kpad=None):
    return U.QTensorDesc(codes, scales, rows, k, (k + 15) // 16 * 16 if kpad is None else kpad,
                         grid, rht, mask, 0)


def gated(x=None, w=None, **kw):
    a = dict(act=F.ACT_SILU, groups=1, off=None, dt=BF16, y=A, ldy=16, gu=A, ldg=32)
    a.update(kw)
    x, w = x or operand(8), w or operand(32)
    return F.lib().ufp4_gated_gemm(ctypes.byref(x), ctypes.byref(w), *a.values(), None)


@pytest.mark.parametrize("x,w,kw,expect", [
    (None, None, dict(act=F.ACT_NONE), -1), (None, None, dict(act=3), -1),
    (None, None, dict(dt=2), -1), (None, None, dict(y=None), -1), (None, None, dict(y=A + 1), -1),
    (None, None, dict(gu=A + 1), -1), (None, None, dict(dt=F32, gu=A + 2), -1),
    (operand(8, codes=None), None, {}, -1), (None, operand(32, scales=A + 8), {}, -1),
    (operand(0), None, {}, -2), (None, operand(31), {}, -2),
    (None, operand(34), dict(groups=4, off=A), -2), (None, None, dict(groups=2), -2),
    (None, None, dict(groups=0), -2), (None, None, dict(groups=1025, off=A), -2),
    (None, None, dict(ldy=15), -2), (None, None, dict(ldg=31), -2),
    (None, None, dict(ldy=1 << 58), -2), (None, None, dict(ldg=1 << 58), -2),
    (operand(8, 80), None, {}, -3), (operand(8, grid=1), None, {}, -3),
    (operand(8, rht=1), None, {}, -3),
    (operand(8, rht=1, mask=1), operand(32, rht=1, mask=2), {}, -3),
    (operand(8, 65537), operand(32, 65537), {}, -4),
])
def test_gated_rejects(x, w, kw, expect):
    assert gated(x, w, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(dy=None), -1), (dict(gu=None), -1), (dict(out=None), -1), (dict(dy=A + 1), -1),
    (dict(gu=A + 1), -1), (dict(out=A + 1), -1), (dict(act=0), -1), (dict(act=9), -1),
    (dict(dt=4), -1), (dict(ldy=63), -2), (dict(ldg=127), -2), (dict(rows=-1), -2),
    (dict(cols=0), -2), (dict(cols=(1 << 23) + 1, ldy=BIG, ldg=BIG), -2),
    (dict(rows=0, dy=None, gu=None, out=None), 0),
])
def test_gated_bwd_rejects(kw, expect):
    a = dict(dy=A, ldy=64, gu=A, ldg=128, act=F.ACT_GELU, dt=BF16, rows=4, cols=64, out=A)
    a.update(kw)
    assert F.lib().ufp4_gated_bwd(*a.values(), None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), -1), (dict(q=None), -1), (dict(s=None), -1), (dict(x=A + 1), -1),
    (dict(q=A + 8), -1), (dict(s=A + 2), -1), (dict(dt=2), -1), (dict(ld=63), -2),
    (dict(rows=-1), -2), (dict(cols=0), -2), (dict(rows=0, x=None, q=None, s=None), 0),
])
def test_int8_quantize_rejects(kw, expect):
    a = dict(x=A, ld=64, dt=BF16, rows=4, cols=64, q=A, s=A)
    a.update(kw)
    assert F.lib().ufp4_int8_quantize(*a.values(), None) == expect


def rows(**kw):
    a = dict(q=A, scale=A, rows=32, k=64)
    a.update(kw)
    return Rows(*a.values())


# w, bias, act, groups, offsets, type, y, ld: what both products take
PRODUCT = [
    (dict(w=rows(q=None)), -1), (dict(w=rows(scale=None)), -1), (dict(w=rows(q=A + 8)), -1),
    (dict(w=rows(scale=A + 2)), -1), (dict(bias=A + 2), -1), (dict(act=3), -1),
    (dict(act=-1), -1), (dict(dt=2), -1), (dict(y=None), -1), (dict(y=A + 1), -1),
    (dict(off=A + 4, groups=2), -1), (dict(groups=2), -2), (dict(groups=0, off=A), -2),
    (dict(groups=1025, off=A), -2), (dict(groups=3, off=A), -2),
    (dict(w=rows(rows=0)), -2), (dict(w=rows(k=63)), -2),
    (dict(w=rows(rows=33), act=F.ACT_SILU), -2), (dict(w=rows(rows=34), groups=2, off=A, act=1), -2),
    (dict(w=rows(rows=(1 << 24) + 2), ldy=BIG), -2), (dict(ldy=31), -2), (dict(act=1, ldy=15), -2),
    (dict(m=-1), -2), (dict(m=1 << 30, ldy=1 << 31), -2), (dict(m=0, y=None), 0),
    (dict(k=131072), -4),
]


@pytest.mark.parametrize("kw,expect", PRODUCT)
@pytest.mark.parametrize("linear", [False, True])
def test_int8_products_reject(linear, kw, expect):
    a = dict(w=rows(), bias=None, act=0, groups=1, off=None, dt=BF16, y=A, ldy=32)
    m, k = kw.get("m", 8), kw.get("k", 64)
    a.update({n: v for n, v in kw.items() if n not in ("m", "k")})
    if k != 64:
        a["w"] = rows(k=k)
    w = a["w"]                                       # stays alive
    a["w"] = ctypes.addressof(w)
    if linear:
        got = F.lib().ufp4_int8_linear(A, k, BF16, m, k, *a.values(), A, 1 << 30, None)
    else:
        x = rows(rows=m, k=k)
        got = F.lib().ufp4_int8_gemm(ctypes.addressof(x), *a.values(), None)
    assert got == expect


def test_int8_left_operand_and_workspace():
    w = rows()
    L, pw = F.lib(), ctypes.addressof(w)
    tail = (pw, None, 0, 1, None, BF16, A, 32)
    for bad, expect in ((rows(q=None, rows=8), -1), (rows(q=A + 4, rows=8), -1),
                        (rows(scale=None, rows=8), -1), (rows(rows=8, k=65), -2)):
        assert L.ufp4_int8_gemm(ctypes.addressof(bad), *tail, None) == expect
    assert L.ufp4_int8_gemm(None, *tail, None) == -1
    good = rows(rows=8)
    assert L.ufp4_int8_gemm(ctypes.addressof(good), None, *tail[1:], None) == -1
    need = F.ufp4_int8_linear_workspace_size(80, 64)
    assert need >= 80 * 128 + 80 * 4 and F.ufp4_int8_linear_workspace_size(-1, 64) == 0
    assert F.ufp4_int8_linear_workspace_size(8, 64) == 0
    assert F.ufp4_int8_linear_workspace_size(8, 64, grouped=True) >= 8 * 128 + 8 * 4
    lin = lambda x, ld, ws, n: L.ufp4_int8_linear(x, ld, BF16, 80, 64, *tail, ws, n, None)
    assert lin(A, 64, A, need - 1) == -1 and lin(A, 64, None, need) == -1
    assert lin(A, 64, A + 8, need) == -1 and lin(None, 64, A, need) == -1
    assert lin(A + 1, 64, A, need) == -1 and lin(A, 63, A, need) == -2


def test_sizes():
    assert F.int8_kpad(1) == 128 and F.int8_kpad(128) == 128 and F.int8_kpad(129) == 256
    assert F.ufp4_layernorm_bwd_workspace_size(0, 64) >= 2 * 64 * 4
    assert F.ufp4_layernorm_bwd_workspace_size(-1, 64) == 0
    assert F.ufp4_layernorm_bwd_workspace_size(4, 0) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    x, w, f = bf(4, 64), bf(64), torch.zeros(4)
    q = U.Quantized(torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 4)), 4, 64, 64, 0, 0,
                    0)
    r = F.Int8Rows(torch.zeros((4, 128), dtype=torch.int8), f, 64)
    for call in (lambda: F.ufp4_layernorm(x, w), lambda: F.ufp4_layernorm_bwd(x, x, w, f, f),
                 lambda: F.ufp4_dropout(x, 0.1, 0), lambda: F.ufp4_gated_gemm(q, q),
                 lambda: F.ufp4_gated_bwd(bf(4, 32), x), lambda: F.ufp4_int8_quantize(x),
                 lambda: F.ufp4_int8_gemm(r, r), lambda: F.ufp4_int8_linear(x, r)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: F.ufp4_layernorm(x.double(), w), lambda: F.ufp4_dropout(x.half(), 0.1, 0),
                 lambda: F.ufp4_gated_bwd(bf(4, 32), x.half()),
                 lambda: F.ufp4_int8_quantize(x.half()),
                 lambda: F.ufp4_gated_gemm(q, q, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()


def test_the_tensors_device_is_current(monkeypatch):
    """As of the block operators."""
    at, seen = [0], []

    @contextlib.contextmanager
    def device(d):
        before, at[0] = at[0], d.index
        try:
            yield
        finally:
            at[0] = before

    monkeypatch.setattr(B, "_current_device", lambda: at[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(B, "_raw_stream", lambda index: ("stream of", index))
    monkeypatch.setattr(F, "lib", lambda: types.SimpleNamespace(
        some_call=lambda *a: seen.append((at[0], a)) or 0))
    F._call("some_call", torch.device("cuda", 2), 7)
    assert seen == [(2, (7, ("stream of", 2)))] and at == [0]
    src = open(F.__file__).read()
    for n in F.EXPORTS:
        if not n.endswith("_size"):
            assert f'_call("{n}", ' in src and f"lib().{n}(" not in src, n
