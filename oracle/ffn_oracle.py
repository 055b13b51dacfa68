"""64-bit oracle of the feed-forward operators: layer norm, dropout, the gated
product's activation, rows in int8.  Plain NumPy written from the formulas, on
values that are already of the tensors' types (float arrays); it shares no code
with the GPU path.  Nothing is rounded here except where a definition rounds
(the residual stream; the dropout's and the codes' FP32 operations, which are
reproduced bit for bit)."""
from __future__ import annotations

import math

import numpy as np

from .block_oracle import residual_sum, round_bf16  # noqa: F401
from .ufp4_oracle import philox4x32_10

SILU, GELU = 1, 2


# -- layer norm ---------------------------------------------------------------
def layernorm(h, w, b, eps):
    """(y, mean, rstd, xhat) of rows h; b may be None."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    mean = h.mean(1)
    d = h - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    xhat = d * rstd[:, None]
    return xhat * w + (0.0 if b is None else np.asarray(b, np.float64)), mean, rstd, xhat


def layernorm_bwd(dy, h, w, eps, dh=None):
    """(dx, dw, db)."""
    dy, w = np.asarray(dy, np.float64), np.asarray(w, np.float64)
    _, _, rstd, xhat = layernorm(h, w, None, eps)
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True)
                          - xhat * (g * xhat).mean(1, keepdims=True))
    return dx + (0.0 if dh is None else dh), (dy * xhat).sum(0), dy.sum(0)


# -- dropout ------------------------------------------------------------------
def threshold(p):
    return int(math.floor(p * 65536.0 + 0.5))


def dropout_keep(rows, cols, p, seed, offset, row0=0):
    """bool [rows, cols]: rows row0 .. row0 + rows of a tensor."""
    groups = -(-cols // 8)
    at = np.uint64(row0 * groups) + np.arange(rows * groups, dtype=np.uint64)
    r = np.stack(philox4x32_10(at & np.uint64(0xFFFFFFFF), at >> np.uint64(32),
                               np.uint64(offset & 0xFFFFFFFF), np.uint64(offset >> 32),
                               seed & 0xFFFFFFFF, seed >> 32), 1)
    bits = np.stack([r & 0xFFFF, r >> 16], 2).reshape(rows, groups * 8)[:, :cols]
    return bits >= threshold(p)


def dropout(x, p, seed, offset, res=None, bf16=False):
    """The result's bits: FP32 operations, rounded to the type."""
    t = threshold(p)
    scale = np.float32(65536.0 / (65536 - t)) if t < 65536 else np.float32(0)
    x = np.asarray(x, np.float32)
    keep = dropout_keep(*x.shape, p, seed, offset)
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.where(keep, x * scale, np.float32(0)) if t else x
        if res is not None:
            y = y + np.asarray(res, np.float32)
    return round_bf16(y) if bf16 else y


# -- activations ----------------------------------------------------------------
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(g, kind):
    """(value, slope) of the activation."""
    g = np.asarray(g, np.float64)
    if kind == SILU:
        e = np.exp(-np.abs(g))
        p = np.where(g >= 0, 1.0, e) / (1.0 + e)
        q = np.where(g >= 0, e, 1.0) / (1.0 + e)
        return g * p, p * (1.0 + g * q)
    c = 0.5 * _erfc(-g / math.sqrt(2.0)) if g.size else g
    return g * c, c + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)


def act_error(g, kind, u):
    """Bounds of what FP32 makes of (value, slope), u half a step.  silu: p is
    within 6 u of itself (the exponential and the reciprocal two each, the sum) and
    1.3 |g| u where g < 0, 1 u where g >= 0, for the rounded exponent; 1 - p is off by
    as much of p and u, and three more roundings follow.  gelu: the argument of erfc is off by 2 u of itself (the constant and the
    product), which moves c = erfc / 2 by 2 u |g| phi(g); erfc itself is granted
    6 (1 + g^2 / 2) u for its fit and exponent, 12 u for its reciprocal and
    exponential (two each, at a slope of up to 2) and 4 u for its products, of the
    half h = min(c, 1 - c) that is computed; exp(-g^2 / 2) is off by (1.5 g^2 + 4) u
    of itself, and each product and sum adds u.  What is below the normal numbers may
    be zero."""
    g = np.asarray(g, np.float64)
    value, slope = act(g, kind)
    tiny = 1e-36 * (1.0 + np.abs(g))
    if kind == SILU:
        e = np.exp(-np.abs(g))
        p = np.where(g >= 0, 1.0, e) / (1.0 + e)
        rel = (6 + np.where(g < 0, 1.3 * np.abs(g), 1.0)) * u
        return ((rel + 2 * u) * np.abs(value) + tiny,
                (rel + 4 * u) * p * (1.0 + np.abs(g) * (1.0 - p)) + (rel + u) * p * p * np.abs(g)
                + u * p * np.abs(g) + tiny)
    c = 0.5 * _erfc(-g / math.sqrt(2.0)) if g.size else g
    phi = np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    c_err = 2 * u * np.abs(g) * phi + (22 + 3 * g * g) * u * np.minimum(c, 1 - c) + u * (g > 0)
    return (np.abs(g) * c_err + 2 * u * np.abs(value) + tiny,
            c_err + (1.5 * g * g + 8) * u * np.abs(g) * phi + 2 * u * np.abs(slope) + tiny)


# -- int8 -------------------------------------------------------------------------
def int8_quantize(x):
    """(codes [rows, cols] int64, scales FP32) bit for bit; finite rows, or rows
    that hold an infinity or a NaN: scale NaN, codes 0."""
    x = np.asarray(x, np.float32)
    top = np.abs(x).max(1, initial=0)
    bad = ~np.isfinite(top)
    t = np.where(bad, np.float32(0), top).astype(np.float32)
    lift = np.where(t < np.float32(2.0 ** -64), np.float32(2.0 ** 64),
                    np.where(t > np.float32(2.0 ** 64), np.float32(2.0 ** -64), np.float32(1)))
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        inv = np.where(t > 0, np.float32(127) * (np.float32(1) / (t * lift)), np.float32(0)).astype(np.float32)
        codes = np.rint(np.where(bad[:, None], np.float32(0), x * lift[:, None] * inv[:, None]))
    scale = np.where(bad, np.float32(np.nan), t / np.float32(127)).astype(np.float32)
    return np.where(bad[:, None], 0, codes).astype(np.int64), scale


def int8_product(qa, sa, qw, sw, bias=None):
    """FP32 [M, N] bit for bit: the exact sum, times sa, times sw, plus bias."""
    s = (np.asarray(qa, np.float64) @ np.asarray(qw, np.float64).T).astype(np.int64)
    p = s.astype(np.float32) * np.asarray(sa, np.float32)[:, None]
    p = p * np.asarray(sw, np.float32)[None, :]
    return p if bias is None else p + np.asarray(bias, np.float32)
