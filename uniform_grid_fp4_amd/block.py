"""Binding of the operators around the 4-bit GEMMs (include/ufp4_block.h): RMS
norm with the residual's addition and an optional E4M3 output, the MoE router
with its balance loss, dispatch to and combination from expert order, and the
global gradient norm with clipping.

As in ufp4.py: torch provides device memory (outputs are allocated here unless
given) and the current stream, every step runs in libufp4's HIP kernels, and
there is no fallback.  Tensors of a wrong type raise TypeError, of a wrong
shape, stride or device ValueError; what the library itself refuses raises
UFP4Error.  Nothing here waits for the GPU or copies to the host.
"""
from __future__ import annotations

import ctypes
import operator
from array import array
from itertools import chain
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import ufp4 as U

# Every symbol include/ufp4_block.h declares.
EXPORTS = ("ufp4_rmsnorm", "ufp4_rmsnorm_bwd", "ufp4_rmsnorm_bwd_workspace_size",
           "ufp4_moe_route", "ufp4_moe_route_bwd", "ufp4_moe_route_workspace_size",
           "ufp4_moe_dispatch", "ufp4_moe_dispatch_bwd", "ufp4_moe_combine",
           "ufp4_moe_combine_bwd", "ufp4_grad_norm", "ufp4_grad_clip",
           "ufp4_grad_norm_workspace_size")
MAX_EXPERTS, MAX_CHOICES = 1024, 16
E4M3 = torch.float8_e4m3fn
_CODE = U._OUT_CODE                               # element types: float32, bfloat16


_lib = None


def lib() -> ctypes.CDLL:
    """libufp4.so with the block operators' C signatures declared."""
    global _lib
    if _lib is not None and _lib is U._lib:
        return _lib
    L = U.lib()
    P, I64, I32, S = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    R, G = P, P                                      # ufp4_routing, ufp4_grad: arrays of words
    L.ufp4_rmsnorm.argtypes = [P, I64, P, I64, P, I32, I32, I64, I64, ctypes.c_float, P, P, P, P,
                               P, P]
    L.ufp4_rmsnorm_bwd.argtypes = [P, I64, P, I64, P, P, P, I64, I32, I32, I64, I64, P, P, P, S, P]
    L.ufp4_rmsnorm_bwd_workspace_size.argtypes = [I64, I64]
    L.ufp4_moe_route.argtypes = [P, I64, I32, P, I64, I32, I32, I32, R, P, S, P]
    L.ufp4_moe_route_bwd.argtypes = [P, I64, I32, I64, I32, I32, I32, R, P, P, P, P]
    L.ufp4_moe_route_workspace_size.argtypes = [I64, I32]
    L.ufp4_moe_dispatch.argtypes = [P, I64, P, I32, I64, I32, I64, P, P]
    L.ufp4_moe_dispatch_bwd.argtypes = [P, P, I32, I64, I32, I64, P, P]
    L.ufp4_moe_combine.argtypes = [P, P, P, P, I64, I32, I64, I32, I64, P, P]
    L.ufp4_moe_combine_bwd.argtypes = [P, I64, P, P, P, I32, I64, I32, I64, P, P, P]
    L.ufp4_grad_norm.argtypes = [G, I64, P, S, P, P]
    L.ufp4_grad_clip.argtypes = [G, I64, P, ctypes.c_double, ctypes.c_double, P]
    L.ufp4_grad_norm_workspace_size.argtypes = []
    for f in EXPORTS:
        getattr(L, f).restype = S if f.endswith("_size") else I32
    _lib = L
    return L


# ---------------------------------------------------------------------------
# Checks
# ---------------------------------------------------------------------------
def _rows2d(t: torch.Tensor, name: str, like: Optional[torch.Tensor] = None) -> int:
    """The row stride of a 2-D tensor with unit column stride, of `like`'s
    shape, type and device when given."""
    if like is not None:
        _like(t, name, like.dtype, like.shape, like.device)
    else:
        if t.dtype not in _CODE:
            raise TypeError(f"{name} is float32 or bfloat16, got {t.dtype}")
        if not t.is_cuda:
            raise ValueError(f"{name} is not on a GPU")
        if t.dim() != 2 or t.shape[1] < 1:
            raise ValueError(f"{name} is 2-D with at least one column, got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.shape[1]
    ld, unit = t.stride()
    if unit != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} needs unit column stride, got strides {t.stride()}")
    # a single row's stride is not used (and may be anything)
    return ld if t.shape[0] > 1 else t.shape[1]


def _like(t: torch.Tensor, name: str, dtype, shape, device) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name} is {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _exact(t: torch.Tensor, name: str, dtype, shape, device) -> torch.Tensor:
    """t, contiguous and of that type, shape and device."""
    _like(t, name, dtype, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    return t


def _weight(w: torch.Tensor, x: torch.Tensor) -> int:
    if w.dtype not in (x.dtype, torch.float32):
        raise TypeError(f"weight is {x.dtype} or float32, got {w.dtype}")
    _exact(w, "weight", w.dtype, (x.shape[1],), x.device)
    return _CODE[w.dtype]


def _new(like: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of that shape and type (empty_like is the cheapest
    allocation, but keeps strides)."""
    return torch.empty_like(like) if like.is_contiguous() else like.new_empty(like.shape)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# torch.cuda.current_stream(device).cuda_stream without the Stream object (2 us
# a call, a tenth of a single-token norm's time).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
# torch.cuda.current_device() without its check that torch has set up the GPUs.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(device: torch.device):
    return _raw_stream(device.index)


def _call(name: str, device: torch.device, *args):
    """As ufp4._call, for the calls whose host time counts."""
    index = device.index
    if index == _current_device():
        st = getattr(lib(), name)(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = getattr(lib(), name)(*args, _raw_stream(index))
    if st:
        U._check(st, name)


# Tells autograd that a tensor, or each of a list, was written in place.
_written = torch.autograd.graph.increment_version


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------
class NormOut(NamedTuple):
    """y (None unless asked for), h = x + residual (x itself without one), rstd
    FP32 [rows], and with q8 the E4M3 rows q and their FP32 scales
    (y ~ q * scale[:, None]), else None."""
    y: Optional[torch.Tensor]
    h: torch.Tensor
    rstd: torch.Tensor
    q: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]


def ufp4_rmsnorm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, y: bool = True, q8: bool = False,
                 out_h: Optional[torch.Tensor] = None) -> NormOut:
    """RMS norm of x (+ residual), 2-D bf16 or float32 with any row stride; the
    weight is of x's type or float32.  `y` and `q8` choose the outputs: the
    input's type, and E4M3 with one scale per row (max |y| / 448).  `out_h`
    receives the sum and may be x or residual itself (in place)."""
    ld = _rows2d(x, "x")
    wd = _weight(weight, x)
    rows, cols = x.shape
    dev = x.device
    ldr, h = 0, x
    if residual is not None:
        ldr = _rows2d(residual, "residual", x)
        h = _new(x) if out_h is None else \
            _exact(out_h, "out_h", x.dtype, (rows, cols), dev)
    elif out_h is not None:
        raise ValueError("out_h is given without a residual")
    out = _new(x) if y else None
    q = scale = None
    if q8:
        q = torch.empty((rows, cols), dtype=E4M3, device=dev)
        rstd, scale = torch.empty((2, rows), dtype=torch.float32, device=dev).unbind(0)
    else:
        rstd = torch.empty((rows,), dtype=torch.float32, device=dev)
    _call("ufp4_rmsnorm", dev, _p(x), ld, _p(residual), ldr, _p(weight), _CODE[x.dtype], wd, rows,
          cols, eps, _p(h) if residual is not None else None, _p(out), _p(q), _p(scale), _p(rstd))
    if out_h is not None:
        _written(out_h)
    return NormOut(out, h, rstd, q, scale)


def ufp4_rmsnorm_bwd_workspace_size(rows: int, cols: int) -> int:
    return int(lib().ufp4_rmsnorm_bwd_workspace_size(rows, cols))


def ufp4_rmsnorm_bwd(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                     dh: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None
                     ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dw) of ufp4_rmsnorm from dy, the gradient of y, and dh, what
    reaches h from elsewhere (None: nothing).  dx is the gradient of x and of
    the residual; dw has the weight's type."""
    ldh = _rows2d(h, "h")
    ldy = _rows2d(dy, "dy", h)
    ldd = _rows2d(dh, "dh", h) if dh is not None else 0
    wd = _weight(weight, h)
    rows, cols = h.shape
    dev = h.device
    _exact(rstd, "rstd", torch.float32, (rows,), dev)
    dx, dw = _new(h), torch.empty_like(weight)
    ws, nbytes = _workspace(workspace, lib().ufp4_rmsnorm_bwd_workspace_size(rows, cols), dev)
    _call("ufp4_rmsnorm_bwd", dev, _p(dy), ldy, _p(h), ldh, _p(weight), _p(rstd), _p(dh), ldd,
          _CODE[h.dtype], wd, rows, cols, _p(dx), _p(dw), _p(ws), nbytes)
    return dx, dw


def _workspace(given: Optional[torch.Tensor], nbytes: int, device):
    if given is None:
        return torch.empty((nbytes,), dtype=torch.uint8, device=device), nbytes
    if given.device != device or not given.is_contiguous():
        raise ValueError(f"the workspace is contiguous and on {device}")
    return given, given.numel() * given.element_size()


# ---------------------------------------------------------------------------
# Router
# ---------------------------------------------------------------------------
class Routing(NamedTuple):
    """What the router decides (see ufp4_routing in include/ufp4_block.h).
    `offsets` is what UFP4ExpertLinear and the grouped GEMMs take over
    tokens * k rows, `slots` what dispatch and combine take."""
    experts: torch.Tensor      # int32 [tokens, k], -1 where there is no choice
    gates: torch.Tensor        # float32 [tokens, k]
    slots: torch.Tensor        # int32 [tokens, k], ~row where there is no choice
    lse: torch.Tensor          # float32 [tokens]
    counts: torch.Tensor       # int64 [experts]
    offsets: torch.Tensor      # int64 [experts + 1]
    n_tokens: torch.Tensor     # int64 [1]
    losses: torch.Tensor       # float32 [2]: balance, z
    renorm: bool

    def words(self) -> array:
        """ufp4_routing: the eight pointers."""
        return array("Q", map(torch.Tensor.data_ptr, self[:8]))


def ufp4_moe_route_workspace_size(tokens: int, n_experts: int) -> int:
    return int(lib().ufp4_moe_route_workspace_size(tokens, n_experts))


def ufp4_moe_route(logits: torch.Tensor, k: int, valid: Optional[torch.Tensor] = None,
                   renorm: bool = True, workspace: Optional[torch.Tensor] = None) -> Routing:
    """Route each token to the k experts of its largest logits (2-D, float32 or
    bf16).  `valid` (bool [tokens]) leaves padding tokens out; `renorm` makes a
    token's gates sum to one, else they are the softmax probabilities."""
    ld = _rows2d(logits, "logits")
    t, e = logits.shape
    dev = logits.device
    if valid is not None:
        _exact(valid, "valid", torch.bool, (t,), dev)
    if not 1 <= k <= min(e, MAX_CHOICES):
        raise ValueError(f"k = {k}: 1 to {MAX_CHOICES} choices of at most {e} experts")
    i32, f32, i64 = torch.int32, torch.float32, torch.int64
    # the whole-number outputs of a type share one allocation (a view costs a
    # third of one)
    experts, slots = torch.empty((2, t, k), dtype=i32, device=dev).unbind(0)
    counts, offsets, n_tokens = torch.empty((2 * e + 2,), dtype=i64,
                                            device=dev).split((e, e + 1, 1))
    r = Routing(experts, torch.empty((t, k), dtype=f32, device=dev), slots,
                torch.empty((t,), dtype=f32, device=dev), counts, offsets, n_tokens,
                torch.empty((2,), dtype=f32, device=dev), bool(renorm))
    need = lib().ufp4_moe_route_workspace_size(t, e)
    ws, nbytes = (None, 0) if need == 0 else _workspace(workspace, need, dev)
    d = r.words()
    _call("ufp4_moe_route", dev, _p(logits), ld, _CODE[logits.dtype], _p(valid), t, e, k,
          int(renorm), d.buffer_info()[0], _p(ws), nbytes)
    return r


def ufp4_moe_route_bwd(logits: torch.Tensor, r: Routing, d_gates: Optional[torch.Tensor] = None,
                       d_losses: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of the logits given to ufp4_moe_route, from that of the
    gates (float32 [tokens, k]) and of the losses (float32 [2], on the GPU)."""
    ld = _rows2d(logits, "logits")
    t, e = logits.shape
    dev = logits.device
    k = r.experts.shape[1]
    _exact(r.experts, "experts", torch.int32, (t, k), dev)
    _exact(r.gates, "gates", torch.float32, (t, k), dev)
    _exact(r.lse, "lse", torch.float32, (t,), dev)
    _exact(r.counts, "counts", torch.int64, (e,), dev)
    _exact(r.n_tokens, "n_tokens", torch.int64, (1,), dev)
    if d_gates is not None:
        _exact(d_gates, "d_gates", torch.float32, (t, k), dev)
    if d_losses is not None:
        _exact(d_losses, "d_losses", torch.float32, (2,), dev)
    out = _new(logits)
    d = r.words()
    _call("ufp4_moe_route_bwd", dev, _p(logits), ld, _CODE[logits.dtype], t, e, k, int(r.renorm),
          d.buffer_info()[0], _p(d_gates), _p(d_losses), _p(out))
    return out


# ---------------------------------------------------------------------------
# Dispatch and combine
# ---------------------------------------------------------------------------
def _slots(slots: torch.Tensor, tokens: Optional[int], device) -> Tuple[int, int]:
    if slots.dim() != 2:
        raise ValueError(f"slots is [tokens, k], got {tuple(slots.shape)}")
    t, k = slots.shape
    _exact(slots, "slots", torch.int32, (t if tokens is None else tokens, k), device)
    if not 1 <= k <= MAX_CHOICES:
        raise ValueError(f"k = {k}: 1 to {MAX_CHOICES} choices")
    return t, k


def _expert_rows(xs: torch.Tensor, name: str, slots: torch.Tensor) -> Tuple[int, int, int]:
    """(tokens, k, columns) of a dense [tokens * k, columns] tensor."""
    ld = _rows2d(xs, name)
    t, k = _slots(slots, None, xs.device)
    rows, cols = xs.shape
    if rows != t * k or ld != cols:
        raise ValueError(f"{name} is dense [{t * k}, columns], got {tuple(xs.shape)} with strides "
                         f"{xs.stride()}")
    return t, k, cols


def _token_rows(t: torch.Tensor, name: str, shape, like: torch.Tensor) -> int:
    """The row stride of a tensor of `shape` and of `like`'s type and device."""
    _like(t, name, like.dtype, shape, like.device)
    return _rows2d(t, name)


def ufp4_moe_dispatch(x: torch.Tensor, slots: torch.Tensor) -> torch.Tensor:
    """x [tokens, cols] to expert order, [tokens * k, cols]; rows without a
    choice are zero."""
    ld = _rows2d(x, "x")
    t, k = _slots(slots, x.shape[0], x.device)
    cols = x.shape[1]
    xs = x.new_empty((t * k, cols))
    _call("ufp4_moe_dispatch", x.device, _p(x), ld, _p(slots), _CODE[x.dtype], t, k, cols, _p(xs))
    return xs


def ufp4_moe_dispatch_bwd(dxs: torch.Tensor, slots: torch.Tensor) -> torch.Tensor:
    """The gradient of dispatch's input: each token's sum over its choices."""
    t, k, cols = _expert_rows(dxs, "dxs", slots)
    dx = dxs.new_empty((t, cols))
    _call("ufp4_moe_dispatch_bwd", dxs.device, _p(dxs), _p(slots), _CODE[dxs.dtype], t, k, cols,
          _p(dx))
    return dx


def ufp4_moe_combine(ys: torch.Tensor, slots: torch.Tensor, gates: torch.Tensor,
                     residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """residual + the gate-weighted sum of each token's rows of ys."""
    t, k, cols = _expert_rows(ys, "ys", slots)
    _exact(gates, "gates", torch.float32, (t, k), ys.device)
    ldr = 0
    if residual is not None:
        ldr = _token_rows(residual, "residual", (t, cols), ys)
    y = ys.new_empty((t, cols))
    _call("ufp4_moe_combine", ys.device, _p(ys), _p(slots), _p(gates), _p(residual), ldr,
          _CODE[ys.dtype], t, k, cols, _p(y))
    return y


def ufp4_moe_combine_bwd(dy: torch.Tensor, ys: torch.Tensor, slots: torch.Tensor,
                         gates: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dys, d_gates) of ufp4_moe_combine; dy itself is the residual's
    gradient."""
    t, k, cols = _expert_rows(ys, "ys", slots)
    ldy = _token_rows(dy, "dy", (t, cols), ys)
    _exact(gates, "gates", torch.float32, (t, k), ys.device)
    dys = torch.empty_like(ys)
    dg = torch.empty_like(gates)
    _call("ufp4_moe_combine_bwd", ys.device, _p(dy), ldy, _p(ys), _p(slots), _p(gates),
          _CODE[ys.dtype], t, k, cols, _p(dys), _p(dg))
    return dys, dg


# ---------------------------------------------------------------------------
# Gradient norm and clipping
# ---------------------------------------------------------------------------
def _dense(t: torch.Tensor) -> bool:
    """Whether t's elements fill one stretch of memory, in any order."""
    if t.is_contiguous():
        return True
    n = 1
    for stride, size in sorted((st, sz) for st, sz in zip(t.stride(), t.shape) if sz != 1):
        if stride != n:
            return False
        n *= size
    return True


_T = torch.Tensor
_dtype_of = operator.attrgetter("dtype")
_PAIR = (0, 1 | 1 << 32)                          # a type and the same type as the output


def _codes(tensors, name):
    try:
        return list(map(_CODE.__getitem__, map(_dtype_of, tensors)))
    except KeyError as e:
        raise TypeError(f"{name} are float32 or bfloat16, got {e.args[0]}") from None


def _grad_list(tensors, out):
    """(descriptors, count, device) of a list of dense tensors.  Lists hold
    hundreds of small tensors and this is most of their call's time, so every
    check runs over the whole list at once."""
    n = len(tensors)
    if n == 0:
        raise ValueError("no tensors")
    codes = _codes(tensors, "tensors")
    gpu = set(map(_T.get_device, tensors))
    if len(gpu) != 1 or -1 in gpu:
        raise ValueError("the tensors are on one GPU")
    plain = all(map(_T.is_contiguous, tensors))
    if not plain and not all(map(_dense, tensors)):
        raise ValueError("a tensor is not dense in memory")
    data, sizes = list(map(_T.data_ptr, tensors)), list(map(_T.numel, tensors))
    ends, types = data, map(_PAIR.__getitem__, codes)
    if out is not None:
        if len(out) != n:
            raise ValueError(f"{len(out)} outputs for {n} tensors")
        ocodes = _codes(out, "outputs")
        if ocodes != codes:
            types = [c | o << 32 for c, o in zip(codes, ocodes)]
        if list(map(_T.numel, out)) != sizes:
            raise ValueError("an output has another size than its tensor")
        if set(map(_T.get_device, out)) != gpu:
            raise ValueError("the outputs are on the tensors' GPU")
        if not (plain and all(map(_T.is_contiguous, out))) and \
                any(o.shape != t.shape or o.stride() != t.stride() for o, t in zip(out, tensors)):
            raise ValueError("an output has another shape or other strides than its tensor")
        ends = list(map(_T.data_ptr, out))
    # ufp4_grad is four 64-bit words, the two types in the last
    words = array("Q", chain.from_iterable(zip(data, ends, sizes, types)))
    return words, n, tensors[0].device


def _norm_of(d, n, dev, workspace):
    norm = torch.empty((), dtype=torch.float32, device=dev)
    ws, nbytes = _workspace(workspace, lib().ufp4_grad_norm_workspace_size(), dev)
    _call("ufp4_grad_norm", dev, d.buffer_info()[0], n, _p(ws), nbytes, _p(norm))
    return norm


def ufp4_grad_norm(tensors: Sequence[torch.Tensor],
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The 2-norm over all elements of all tensors (bf16 or float32, dense), a
    float32 scalar on the GPU."""
    d, n, dev = _grad_list(tensors, None)
    return _norm_of(d, n, dev, workspace)


def ufp4_clip_grads(tensors: Sequence[torch.Tensor], max_norm: float,
                    out: Optional[Sequence[torch.Tensor]] = None, eps: float = 1e-6,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Scale all tensors by min(1, max_norm / (norm + eps)), in place or into
    `out` (as many elements each, contiguous, or of the tensors' shapes and
    strides; bf16 or float32), and return the norm before it.  No two outputs may
    overlap, nor an output another tensor.  The coefficient stays on the GPU:
    nothing waits."""
    d, n, dev = _grad_list(tensors, out)
    norm = _norm_of(d, n, dev, workspace)
    _call("ufp4_grad_clip", dev, d.buffer_info()[0], n, _p(norm), max_norm, eps)
    if out is None:
        _written(tensors)
    return norm
