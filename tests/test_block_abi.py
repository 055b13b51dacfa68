"""The block operators' C ABI without a GPU: every function that
include/ufp4_block.h declares is exported, bad arguments are refused on the
host before anything is enqueued, and the binding refuses tensors of wrong
types, shapes, strides or devices."""
import ctypes
import os
import re

import pytest
import torch

from uniform_grid_fp4_amd import block as B
from uniform_grid_fp4_amd import ufp4 as U

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16 = U.OUT_F32, U.OUT_BF16
A = 0x10000                # an address that is never dereferenced
BIG = 1 << 40


class RoutingDesc(ctypes.Structure):
    """Mirror of ufp4_routing."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("experts", "gates", "slots", "lse", "counts",
                                               "offsets", "n_tokens", "losses")]


class GradDesc(ctypes.Structure):
    """Mirror of ufp4_grad."""
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


def test_library_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "ufp4_block.h")).read()
    decl = sorted(set(re.findall(r"^(?:ufp4_status|size_t)\s+(ufp4_\w+)\(", src, re.M)))
    assert sorted(B.EXPORTS) == decl
    for name in decl:
        assert hasattr(B.lib(), name), name


def norm(**kw):
    a = dict(x=A, ld=64, res=A, ldr=64, w=A, dt=BF16, wdt=BF16, rows=4, cols=64, eps=1e-6, h=A,
             y=A, q=A, scale=A, rstd=A)
    a.update(kw)
    return B.lib().ufp4_rmsnorm(a["x"], a["ld"], a["res"], a["ldr"], a["w"], a["dt"], a["wdt"],
                                a["rows"], a["cols"], a["eps"], a["h"], a["y"], a["q"],
                                a["scale"], a["rstd"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(h=None), -1), (dict(rstd=None), -1),
    (dict(y=None, q=None, scale=None), -1), (dict(q=None), -1), (dict(scale=None), -1),
    (dict(x=A + 1), -1), (dict(res=A + 1), -1), (dict(h=A + 1), -1), (dict(y=A + 1), -1),
    (dict(w=A + 1), -1), (dict(scale=A + 2), -1), (dict(rstd=A + 2), -1),
    (dict(dt=2), -1), (dict(wdt=3), -1), (dict(dt=F32, wdt=BF16), -1),
    (dict(dt=F32, wdt=F32, x=A + 2), -1),
    (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(rows=-1), -2), (dict(cols=0), -2), (dict(ld=63), -2), (dict(ldr=63), -2),
    (dict(cols=(1 << 24) + 1, ld=BIG, ldr=BIG), -2), (dict(rows=(1 << 40) + 1), -2),
    (dict(rows=1 << 40, cols=1 << 24, ld=BIG, ldr=BIG), -2),   # the product passes 63 bits
    (dict(rows=0, x=None, h=None, rstd=None), 0),          # nothing to do
])
def test_rmsnorm_rejects(kw, expect):
    assert norm(**kw) == expect


def norm_bwd(**kw):
    a = dict(dy=A, ldy=64, h=A, ldh=64, w=A, rstd=A, dh=A, ldd=64, dt=BF16, wdt=BF16, rows=4,
             cols=64, dx=A, dw=A, ws=A, n=1 << 20)
    a.update(kw)
    return B.lib().ufp4_rmsnorm_bwd(a["dy"], a["ldy"], a["h"], a["ldh"], a["w"], a["rstd"],
                                    a["dh"], a["ldd"], a["dt"], a["wdt"], a["rows"], a["cols"],
                                    a["dx"], a["dw"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dy=None), -1), (dict(h=None), -1), (dict(w=None), -1), (dict(rstd=None), -1),
    (dict(dx=None), -1), (dict(dw=None), -1), (dict(ws=None), -1), (dict(n=0), -1),
    (dict(ws=A + 8), -1), (dict(dy=A + 1), -1), (dict(dh=A + 1), -1), (dict(dx=A + 1), -1),
    (dict(dw=A + 1), -1), (dict(dt=7), -1), (dict(dt=F32, wdt=BF16), -1),
    (dict(ldy=3), -2), (dict(ldh=3), -2), (dict(ldd=3), -2), (dict(cols=-1), -2),
    (dict(rows=-2), -2), (dict(rows=1 << 40, cols=1 << 24, ldy=BIG, ldh=BIG, ldd=BIG), -2),
])
def test_rmsnorm_bwd_rejects(kw, expect):
    assert norm_bwd(**kw) == expect


def routing(**kw):
    a = {n: A for n, _ in RoutingDesc._fields_}
    a.update(kw)
    return RoutingDesc(**a)


def route(bwd=False, r=None, **kw):
    a = dict(x=A, ld=64, dt=F32, valid=None, t=8, e=64, k=4, renorm=1, ws=A, n=1 << 20, dg=None,
             dl=None, out=A)
    a.update(kw)
    r = r if r is not None else routing()
    ref = ctypes.addressof(r)
    if bwd:
        return B.lib().ufp4_moe_route_bwd(a["x"], a["ld"], a["dt"], a["t"], a["e"], a["k"],
                                          a["renorm"], ref, a["dg"], a["dl"], a["out"], None)
    return B.lib().ufp4_moe_route(a["x"], a["ld"], a["dt"], a["valid"], a["t"], a["e"], a["k"],
                                  a["renorm"], ref, a["ws"], a["n"], None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), -1), (dict(x=A + 2), -1), (dict(dt=5), -1), (dict(renorm=2), -1),
    (dict(ld=63), -2), (dict(t=-1), -2), (dict(e=0), -2), (dict(k=0), -2), (dict(k=65), -2),
    (dict(e=1025, ld=1025), -4), (dict(k=17), -4), (dict(t=1 << 29), -4),
    (dict(r=routing(experts=0)), -1), (dict(r=routing(gates=A + 2)), -1),
    (dict(r=routing(lse=0)), -1), (dict(r=routing(counts=A + 4)), -1),
    (dict(r=routing(n_tokens=0)), -1),
])
def test_route_rejects(bwd, kw, expect):
    assert route(bwd, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(r=routing(slots=0)), -1), (dict(r=routing(offsets=A + 4)), -1),
    (dict(r=routing(losses=0)), -1), (dict(t=65, ws=None), -1), (dict(t=65, ws=A + 8), -1),
    (dict(t=65, n=16), -1),
])
def test_route_forward_only_rejects(kw, expect):
    assert route(False, **kw) == expect


@pytest.mark.parametrize("kw", [dict(dg=A + 2), dict(dl=A + 1), dict(out=None), dict(out=A + 2)])
def test_route_bwd_only_rejects(kw):
    assert route(True, **kw) == -1


def test_route_workspace_size():
    size = B.ufp4_moe_route_workspace_size
    assert size(0, 8) == size(64, 8) == 0           # one workgroup keeps everything in LDS
    assert size(129, 8) > size(65, 8) > 0
    assert size(-1, 8) == 0 and size(8, 0) == 0 and size(8, 1025) == 0


@pytest.mark.parametrize("kw,expect", [
    (dict(a=None), -1), (dict(slots=None), -1), (dict(out=None), -1), (dict(a=A + 1), -1),
    (dict(slots=A + 2), -1), (dict(out=A + 1), -1), (dict(dt=4), -1),
    (dict(t=-1), -2), (dict(k=0), -2), (dict(cols=0), -2), (dict(ld=31), -2),
    (dict(k=17), -4), (dict(t=(1 << 31) // 4), -4), (dict(t=0, a=None, slots=None, out=None), 0),
])
def test_exchange_rejects(kw, expect):
    a = dict(a=A, slots=A, out=A, dt=BF16, t=4, k=4, cols=32, ld=32)
    a.update(kw)
    L = B.lib()
    args = (a["dt"], a["t"], a["k"], a["cols"], a["out"])
    assert L.ufp4_moe_dispatch(a["a"], a["ld"], a["slots"], *args, None) == expect
    assert L.ufp4_moe_combine(a["a"], a["slots"], A, A, a["ld"], *args, None) == expect
    assert L.ufp4_moe_combine_bwd(A, a["ld"], a["a"], a["slots"], A, *args, A, None) == expect
    if "ld" not in kw:
        assert L.ufp4_moe_dispatch_bwd(a["a"], a["slots"], *args, None) == expect


def test_exchange_rejects_bad_gates():
    L = B.lib()
    assert L.ufp4_moe_combine(A, A, None, None, 0, BF16, 4, 4, 32, A, None) == -1
    assert L.ufp4_moe_combine(A, A, A + 2, None, 0, BF16, 4, 4, 32, A, None) == -1
    assert L.ufp4_moe_combine(A, A, A, A + 1, 32, BF16, 4, 4, 32, A, None) == -1
    assert L.ufp4_moe_combine_bwd(A, 32, A, A, A, BF16, 4, 4, 32, A, None, None) == -1
    assert L.ufp4_moe_combine_bwd(A + 1, 32, A, A, A, BF16, 4, 4, 32, A, A, None) == -1


def grad(**kw):
    a = dict(data=A, out=A, n=8, dtype=F32, out_dtype=F32)
    a.update(kw)
    return GradDesc(*a.values())


@pytest.mark.parametrize("g,norm_status,clip_status", [
    (grad(data=None), -1, -1), (grad(data=A + 2), -1, -1), (grad(dtype=9), -1, -1),
    (grad(n=-1), -2, -2), (grad(n=(1 << 44) + 1), -2, -2),
    (grad(out=None), None, -1), (grad(out=A + 1), None, -1), (grad(out_dtype=2), None, -1),
    (grad(dtype=BF16), None, -1),                   # in place with two types
])
def test_grads_reject(g, norm_status, clip_status):
    L = B.lib()
    d = (GradDesc * 2)(grad(), g)
    p = ctypes.addressof(d)
    if norm_status is not None:
        assert L.ufp4_grad_norm(p, 2, A, 1 << 20, A, None) == norm_status
    assert L.ufp4_grad_clip(p, 2, A, 1.0, 1e-6, None) == clip_status


def test_grad_call_arguments():
    L = B.lib()
    p = ctypes.addressof((GradDesc * 1)(grad()))
    n = int(L.ufp4_grad_norm_workspace_size())
    assert L.ufp4_grad_norm(p, -1, A, n, A, None) == -2
    assert L.ufp4_grad_norm(None, 1, A, n, A, None) == -1
    assert L.ufp4_grad_norm(p, 1, None, n, A, None) == -1
    assert L.ufp4_grad_norm(p, 1, A, n - 1, A, None) == -1
    assert L.ufp4_grad_norm(p, 1, A, n, None, None) == -1
    for max_norm, eps in ((-1.0, 0.0), (float("nan"), 0.0), (1.0, -1e-6), (1.0, float("nan"))):
        assert L.ufp4_grad_clip(p, 1, A, max_norm, eps, None) == -1
    assert L.ufp4_grad_clip(p, 1, None, 1.0, 0.0, None) == -1


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    slots = torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: B.ufp4_rmsnorm(x, w), lambda: B.ufp4_moe_route(x, 2),
                 lambda: B.ufp4_moe_dispatch(x, slots), lambda: B.ufp4_grad_norm([x]),
                 lambda: B.ufp4_moe_dispatch_bwd(torch.zeros((8, 64)), slots),
                 lambda: B.ufp4_rmsnorm_bwd(x, x, w, torch.zeros(4)),
                 lambda: B.ufp4_clip_grads([], 1.0)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: B.ufp4_rmsnorm(x.double(), w), lambda: B.ufp4_moe_route(x.half(), 2),
                 lambda: B.ufp4_grad_norm([x.half()])):
        with pytest.raises(TypeError):
            call()


def test_dense_storage_orders():
    """What the clipping calls take as one stretch of memory."""
    t = torch.zeros((3, 4, 5))
    assert B._dense(t) and B._dense(t.permute(2, 0, 1)) and B._dense(t[1]) and B._dense(t[:, :1][:1])
    assert not B._dense(t[:, 1:]) and not B._dense(t[..., 0]) and not B._dense(
        torch.zeros(1).expand(7))
    assert B._dense(torch.zeros((0, 3))) and B._dense(torch.zeros(()))
