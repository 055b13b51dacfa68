"""Binding of the operators of a feed-forward sublayer (include/ufp4_ffn.h):
layer norm with the residual's addition, the gated product of two projections
on 4-bit operands, dropout from a counter-based generator, and rows in 8-bit
integers with their product.

As in block.py: torch provides device memory and the current stream, every step
runs in libufp4's HIP kernels, and there is no fallback.  Tensors of a wrong
type raise TypeError, of a wrong shape, stride or device ValueError; what the
library itself refuses raises UFP4Error.  Nothing here waits for the GPU or
copies to the host.
"""
from __future__ import annotations

import ctypes
from array import array
from typing import NamedTuple, Optional, Tuple, Union

import torch

from . import block as B
from . import ufp4 as U
from .block import _CODE, _exact, _like, _new, _p, _rows2d, _workspace, _written

# Every symbol include/ufp4_ffn.h declares.
EXPORTS = ("ufp4_layernorm", "ufp4_layernorm_bwd", "ufp4_layernorm_bwd_workspace_size",
           "ufp4_dropout", "ufp4_gated_gemm", "ufp4_gated_bwd", "ufp4_int8_quantize",
           "ufp4_int8_gemm", "ufp4_int8_linear", "ufp4_int8_linear_workspace_size")
ACT_NONE, ACT_SILU, ACT_GELU = 0, 1, 2
MAX_GROUPS = 1024
INT8_MAX_K = 131071
INT8_FEW_COLUMNS = 16384      # beyond, few rows too are quantized into a workspace,
INT8_FEW_ELEMENTS = 2048      # from so many on

_lib = None


def lib() -> ctypes.CDLL:
    """libufp4.so with the feed-forward operators' C signatures declared."""
    global _lib
    if _lib is not None and _lib is U._lib:
        return _lib
    L = U.lib()
    P, I64, I32, S = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    U64, F32, F64 = ctypes.c_uint64, ctypes.c_float, ctypes.c_double
    Q = ctypes.POINTER(U.QTensorDesc)
    R = P                                            # ufp4_int8_rows: four words
    L.ufp4_layernorm.argtypes = [P, I64, P, I64, P, P, I32, I32, I64, I64, F32, P, P, P, P, P]
    L.ufp4_layernorm_bwd.argtypes = [P, I64, P, I64, P, P, P, P, I64, I32, I32, I64, I64, P, P, P,
                                     P, S, P]
    L.ufp4_layernorm_bwd_workspace_size.argtypes = [I64, I64]
    L.ufp4_dropout.argtypes = [P, I64, P, I64, I32, I64, I64, F64, U64, U64, P, P, P]
    L.ufp4_gated_gemm.argtypes = [Q, Q, I32, I32, P, I32, P, I64, P, I64, P]
    L.ufp4_gated_bwd.argtypes = [P, I64, P, I64, I32, I32, I64, I64, P, P]
    L.ufp4_int8_quantize.argtypes = [P, I64, I32, I64, I64, P, P, P]
    L.ufp4_int8_gemm.argtypes = [R, R, P, I32, I32, P, I32, P, I64, P]
    L.ufp4_int8_linear.argtypes = [P, I64, I32, I64, I64, R, P, I32, I32, P, I32, P, I64, P, S, P]
    L.ufp4_int8_linear_workspace_size.argtypes = [I64, I64, I32]
    for f in EXPORTS:
        getattr(L, f).restype = S if f.endswith("_size") else I32
    _lib = L
    return L


def _call(name: str, device: torch.device, *args):
    """As block._call."""
    index = device.index
    if index == B._current_device():
        st = getattr(lib(), name)(*args, B._raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = getattr(lib(), name)(*args, B._raw_stream(index))
    if st:
        U._check(st, name)


def _rows(t: torch.Tensor, name: str, like: torch.Tensor) -> int:
    """block._rows2d of a tensor like another; dense ones, as most are, take one
    look (these checks are a third of a small call's time)."""
    if t.dtype == like.dtype and t.shape == like.shape and t.device == like.device \
            and t.is_contiguous():
        return t.shape[1]
    return _rows2d(t, name, like)


def _vector(t: torch.Tensor, name: str, dtype, n: int, device) -> torch.Tensor:
    """block._exact of n numbers."""
    if t.dtype == dtype and t.shape == (n,) and t.device == device and t.is_contiguous():
        return t
    return _exact(t, name, dtype, (n,), device)


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------
class LayerNormOut(NamedTuple):
    """y, h = x + residual (x itself without one), and the rows' mean and
    reciprocal standard deviation, float32 [rows]."""
    y: torch.Tensor
    h: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor


def ufp4_layernorm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   residual: Optional[torch.Tensor] = None, eps: float = 1e-5,
                   out_h: Optional[torch.Tensor] = None) -> LayerNormOut:
    """Layer norm of x (+ residual), 2-D bf16 or float32 with any row stride;
    weight and bias are of x's type or both float32.  `out_h` receives the sum
    and may be x or residual itself (in place)."""
    ld = _rows2d(x, "x")
    rows, cols = x.shape
    dev, dtype = x.device, x.dtype
    wtype = weight.dtype
    if wtype != dtype and wtype != torch.float32:
        raise TypeError(f"weight is {dtype} or float32, got {wtype}")
    _vector(weight, "weight", wtype, cols, dev)
    pb = pr = ph = None
    if bias is not None:
        pb = _vector(bias, "bias", wtype, cols, dev).data_ptr()
    ldr, h = 0, x
    if residual is not None:
        ldr = _rows(residual, "residual", x)
        h = _new(x) if out_h is None else _exact(out_h, "out_h", dtype, (rows, cols), dev)
        pr, ph = residual.data_ptr(), h.data_ptr()
    elif out_h is not None:
        raise ValueError("out_h is given without a residual")
    y = _new(x)
    mean, rstd = x.new_empty((2, rows), dtype=torch.float32).unbind(0)
    _call("ufp4_layernorm", dev, x.data_ptr(), ld, pr, ldr, weight.data_ptr(), pb, _CODE[dtype],
          _CODE[wtype], rows, cols, eps, ph, y.data_ptr(), mean.data_ptr(), rstd.data_ptr())
    if out_h is not None:
        _written(out_h)
    return LayerNormOut(y, h, mean, rstd)


def ufp4_layernorm_bwd_workspace_size(rows: int, cols: int) -> int:
    return int(lib().ufp4_layernorm_bwd_workspace_size(rows, cols))


def ufp4_layernorm_bwd(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                       rstd: torch.Tensor, dh: Optional[torch.Tensor] = None, bias: bool = True,
                       workspace: Optional[torch.Tensor] = None
                       ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """(dx, dw, db) of ufp4_layernorm from dy, the gradient of y, and dh, what
    reaches h from elsewhere (None: nothing).  dx is the gradient of x and of
    the residual; dw and db have the weight's type; db is None without `bias`."""
    ldh = _rows2d(h, "h")
    ldy = _rows(dy, "dy", h)
    ldd = _rows(dh, "dh", h) if dh is not None else 0
    rows, cols = h.shape
    dev = h.device
    wtype = weight.dtype
    if wtype != h.dtype and wtype != torch.float32:
        raise TypeError(f"weight is {h.dtype} or float32, got {wtype}")
    wd = _CODE[_vector(weight, "weight", wtype, cols, dev).dtype]
    _vector(mean, "mean", torch.float32, rows, dev)
    _vector(rstd, "rstd", torch.float32, rows, dev)
    dx, dw = _new(h), torch.empty_like(weight)
    db = torch.empty_like(weight) if bias else None
    ws, nbytes = _workspace(workspace, lib().ufp4_layernorm_bwd_workspace_size(rows, cols), dev)
    _call("ufp4_layernorm_bwd", dev, dy.data_ptr(), ldy, h.data_ptr(), ldh, weight.data_ptr(),
          mean.data_ptr(), rstd.data_ptr(), _p(dh), ldd, _CODE[h.dtype], wd, rows, cols,
          dx.data_ptr(), dw.data_ptr(), _p(db), ws.data_ptr(), nbytes)
    return dx, dw, db


# ---------------------------------------------------------------------------
# Dropout
# ---------------------------------------------------------------------------
_WORD = (1 << 64) - 1


def ufp4_dropout(x: torch.Tensor, p: float, seed: int, offset: Union[int, torch.Tensor] = 0,
                 residual: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """residual + x with each element dropped with probability p and the others
    scaled by 1 / (1 - p) (p in whole 65536ths; residual None: no addition).  The
    mask is a function of (seed, offset, row, column): the same call on the
    gradient of the output is the backward pass.  x and residual are 2-D bf16 or
    float32 with any row stride.  `offset` is a number or an int64 tensor of one
    element on the GPU, which is read when the kernel runs.  `out` may be x or
    residual itself (in place)."""
    ld = _rows2d(x, "x")
    rows, cols = x.shape
    dev = x.device
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p = {p}: a probability")
    ldr = 0
    if residual is not None:
        ldr = _rows(residual, "residual", x)
    y = _new(x) if out is None else _exact(out, "out", x.dtype, (rows, cols), dev)
    there = None
    if isinstance(offset, torch.Tensor):
        _like(offset.reshape(-1), "offset", torch.int64, (1,), dev)
        there, offset = offset.data_ptr(), 0
    _call("ufp4_dropout", dev, x.data_ptr(), ld, None if residual is None else residual.data_ptr(),
          ldr, _CODE[x.dtype], rows, cols, p, seed & _WORD, offset & _WORD, there, y.data_ptr())
    if out is not None:
        _written(out)
    return y


# ---------------------------------------------------------------------------
# Gated product on 4-bit operands
# ---------------------------------------------------------------------------
class GatedOut(NamedTuple):
    """y = act(g) * u [rows, ffn], and gu = (g | u) [rows, 2 ffn] for the
    backward pass (None unless kept)."""
    y: torch.Tensor
    gu: Optional[torch.Tensor]


def _operand(q: U.Quantized, name: str, device=None) -> U.QTensorDesc:
    codes, scales, rows, kpad = q.codes, q.scales, q.rows, q.kpad
    dev = codes.device if device is None else device
    if not (codes.is_cuda and codes.device == dev and scales.device == dev
            and codes.dtype == torch.uint8 and scales.dtype == torch.float32
            and codes.shape == (rows, kpad // 2) and scales.shape == (rows, kpad // 16)
            and codes.is_contiguous() and scales.is_contiguous()):
        if not codes.is_cuda:
            raise ValueError(f"{name} is not on a GPU")
        _exact(codes, f"{name}.codes", torch.uint8, (rows, kpad // 2), dev)
        _exact(scales, f"{name}.scales", torch.float32, (rows, kpad // 16), dev)
    return q.desc()


def _groups(offsets: Optional[torch.Tensor], device) -> int:
    """The number of groups that offsets (int64 [groups + 1]) stand for."""
    if offsets is None:
        return 1
    if offsets.dim() != 1 or not 2 <= offsets.shape[0] <= MAX_GROUPS + 1:
        raise ValueError(f"offsets are [groups + 1], 1 to {MAX_GROUPS} groups, got "
                         f"{tuple(offsets.shape)}")
    _exact(offsets, "offsets", torch.int64, offsets.shape, device)
    return offsets.shape[0] - 1


def _rows_per_group(rows: int, groups: int, of: int) -> int:
    """w's rows of a group over `of`."""
    if rows < 1 or rows % (groups * of):
        raise ValueError(f"{rows} rows of w are not {of} equal parts for each of {groups} groups")
    return rows // (groups * of)


def ufp4_gated_gemm(xq: U.Quantized, wq: U.Quantized, act: int = ACT_SILU, keep: bool = True,
                    offsets: Optional[torch.Tensor] = None,
                    out_dtype: torch.dtype = torch.bfloat16) -> GatedOut:
    """act(x Wg^T) * (x Wu^T) of quantized operands.  wq has Wg's rows, then
    Wu's, for each expert of `offsets` (int64 [experts + 1] over x's rows, the
    last entry their number; None: one group).  `keep` returns g and u too, in
    out_dtype (bf16 or float32).  The order of their sums, and so a row's last bits,
    goes by the sizes of the whole call."""
    if out_dtype not in _CODE:
        raise TypeError(f"out_dtype is float32 or bfloat16, got {out_dtype}")
    dx = _operand(xq, "xq")
    dev = xq.codes.device
    dw = _operand(wq, "wq", dev)
    groups = _groups(offsets, dev)
    f = _rows_per_group(wq.rows, groups, 2)
    new = xq.scales.new_empty
    y = new((xq.rows, f), dtype=out_dtype)
    gu = new((xq.rows, 2 * f), dtype=out_dtype) if keep else None
    _call("ufp4_gated_gemm", dev, ctypes.byref(dx), ctypes.byref(dw), act, groups, _p(offsets),
          _CODE[out_dtype], y.data_ptr(), f, None if gu is None else gu.data_ptr(), 2 * f)
    return GatedOut(y, gu)


def ufp4_gated_bwd(dy: torch.Tensor, gu: torch.Tensor, act: int = ACT_SILU,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient (dg | du) of gu from that of y, [rows, 2 ffn], of gu's type:
    dY of the two projections as one product.  `out` may be gu itself."""
    ldg = _rows2d(gu, "gu")
    rows, cols = gu.shape
    if cols % 2:
        raise ValueError(f"gu is [rows, 2 ffn], got {tuple(gu.shape)}")
    _like(dy, "dy", gu.dtype, (rows, cols // 2), gu.device)
    ldy = cols // 2 if dy.is_contiguous() else _rows2d(dy, "dy")
    dgu = _new(gu) if out is None else _exact(out, "out", gu.dtype, (rows, cols), gu.device)
    _call("ufp4_gated_bwd", gu.device, dy.data_ptr(), ldy, gu.data_ptr(), ldg, act,
          _CODE[gu.dtype], rows, cols // 2, dgu.data_ptr())
    if out is not None:
        _written(out)
    return dgu


# ---------------------------------------------------------------------------
# Rows in 8-bit integers, and their product
# ---------------------------------------------------------------------------
def int8_kpad(k: int) -> int:
    return (k + 127) // 128 * 128


class Int8Rows(NamedTuple):
    """Rows of int8 [rows, int8_kpad(k)], zeros past k, and a float32 scale for
    each: q * scale[:, None] is what they stand for."""
    q: torch.Tensor
    scale: torch.Tensor
    k: int


def ufp4_int8_quantize(x: torch.Tensor) -> Int8Rows:
    """2-D bf16 or float32 rows, any row stride, to int8 with a scale each (max
    |x| / 127): activations by token, or a weight by output channel."""
    ld = _rows2d(x, "x")
    rows, cols = x.shape
    q = torch.empty((rows, int8_kpad(cols)), dtype=torch.int8, device=x.device)
    scale = torch.empty((rows,), dtype=torch.float32, device=x.device)
    _call("ufp4_int8_quantize", x.device, _p(x), ld, _CODE[x.dtype], rows, cols, _p(q), _p(scale))
    return Int8Rows(q, scale, cols)


def _int8_operand(r: Int8Rows, name: str, device) -> array:
    """ufp4_int8_rows: two pointers and two sizes."""
    q, scale, k = r
    if not q.is_cuda:
        raise ValueError(f"{name} is not on a GPU")
    if q.dim() != 2 or not 1 <= k or q.shape[1] != int8_kpad(k):
        raise ValueError(f"{name}.q is [rows, {int8_kpad(max(1, k))}] for k = {k}, got "
                         f"{tuple(q.shape)}")
    if not (q.dtype == torch.int8 and q.device == device and q.is_contiguous()):
        _exact(q, f"{name}.q", torch.int8, q.shape, device)
    n = q.shape[0]
    _vector(scale, f"{name}.scale", torch.float32, n, device)
    return array("Q", (q.data_ptr(), scale.data_ptr(), n, k))


def _int8_out(rows: int, w: Int8Rows, bias, act: int, offsets, out_dtype, device):
    """(words of w, groups, y) of a product with `rows` rows."""
    if out_dtype not in _CODE:
        raise TypeError(f"out_dtype is float32 or bfloat16, got {out_dtype}")
    words = _int8_operand(w, "w", device)
    groups = _groups(offsets, device)
    n = w.q.shape[0]
    cols = _rows_per_group(n, groups, 1 if act == ACT_NONE else 2)
    if bias is not None:
        _vector(bias, "bias", torch.float32, n, device)
    return words, groups, w.scale.new_empty((rows, cols), dtype=out_dtype)


def ufp4_int8_gemm(a: Int8Rows, w: Int8Rows, bias: Optional[torch.Tensor] = None,
                   act: int = ACT_NONE, offsets: Optional[torch.Tensor] = None,
                   out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """a w^T with both scales (+ bias, float32), in bf16 or float32.  With an
    `act`, w has gate rows, then up rows, and the result is act(gate) * up.
    `offsets` (int64 [experts + 1] over a's rows, the last entry their number):
    each row meets its own expert's rows of w."""
    dev = a.q.device
    da = _int8_operand(a, "a", dev)
    if a.k != w.k:
        raise ValueError(f"a has rows of {a.k}, w of {w.k}")
    dw, groups, y = _int8_out(a.q.shape[0], w, bias, act, offsets, out_dtype, dev)
    _call("ufp4_int8_gemm", dev, da.buffer_info()[0], dw.buffer_info()[0], _p(bias), act, groups,
          _p(offsets), _CODE[out_dtype], _p(y), y.shape[1])
    return y


def ufp4_int8_linear_workspace_size(rows: int, cols: int, grouped: bool = False) -> int:
    return int(lib().ufp4_int8_linear_workspace_size(rows, cols, int(grouped)))


def ufp4_int8_linear(x: torch.Tensor, w: Int8Rows, bias: Optional[torch.Tensor] = None,
                     act: int = ACT_NONE, offsets: Optional[torch.Tensor] = None,
                     out_dtype: Optional[torch.dtype] = None,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """ufp4_int8_gemm of ufp4_int8_quantize(x) in one call; the result has x's
    type unless out_dtype is given."""
    ld = _rows2d(x, "x")
    rows, cols = x.shape
    dev = x.device
    if cols != w.k:
        raise ValueError(f"x has rows of {cols}, w of {w.k}")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    dw, groups, y = _int8_out(rows, w, bias, act, offsets, out_dtype, dev)
    size = lib().ufp4_int8_linear_workspace_size
    need = size(rows, cols, offsets is not None)
    ws = None
    if need or (y.shape[1] > INT8_FEW_COLUMNS and rows * int8_kpad(cols) >= INT8_FEW_ELEMENTS):
        ws, need = _workspace(workspace, need or size(rows, cols, True), dev)
        ws = ws.data_ptr()
    _call("ufp4_int8_linear", dev, x.data_ptr(), ld, _CODE[x.dtype], rows, cols,
          dw.buffer_info()[0], _p(bias), act, groups, _p(offsets), _CODE[out_dtype], y.data_ptr(),
          y.shape[1], ws, need)
    return y
