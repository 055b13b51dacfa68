"""64-bit oracle of the block operators: RMS norm, MoE router, dispatch and
combine, gradient clipping.  Plain NumPy written from the formulas, on values
that are already of the tensors' types (float arrays); it shares no code with
the GPU path.  Nothing is rounded here except where a definition rounds (the
residual stream)."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def round_bf16(x):
    """float array -> the nearest bf16 values (ties to even) of its FP32 form."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32)


def residual_sum(x, r, bf16):
    s = np.asarray(x, np.float32) + np.asarray(r, np.float32)
    return (round_bf16(s) if bf16 else s).astype(np.float64)


def rmsnorm(h, w, eps):
    """(y, rstd) of rows h."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * w, rstd


def rmsnorm_bwd(dy, h, w, eps, dh=None):
    """(dx, dw, magnitude of dx's terms, sum of |terms| of dw)."""
    dy, h, w = (np.asarray(v, np.float64) for v in (dy, h, w))
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    xhat, g = h * rstd[:, None], dy * w
    mean = (g * xhat).mean(1, keepdims=True)
    dx = rstd[:, None] * (g - xhat * mean)
    size = rstd[:, None] * (np.abs(g) + np.abs(xhat) * np.abs(g * xhat).mean(1, keepdims=True))
    if dh is not None:
        dx, size = dx + dh, size + np.abs(dh)
    return dx, (dy * xhat).sum(0), size, np.abs(dy * xhat).sum(0)


def route(logits, k, valid=None, renorm=True):
    """Dict of the router's outputs, plus p [tokens, experts] (zero rows for
    tokens that take no part).  Finite or -inf logits."""
    x = np.asarray(logits, np.float64)
    t, e = x.shape
    live = np.ones(t, bool) if valid is None else np.asarray(valid, bool).copy()
    live &= ~np.all(np.isneginf(x), axis=1)
    top = np.where(live, x.max(1, initial=-np.inf), 0.0)
    ex = np.where(live[:, None], np.exp(np.where(live[:, None], x, 0.0) - top[:, None]), 0.0)
    sums = ex.sum(1)
    lse = np.where(live, top + np.log(np.where(live, sums, 1.0)), -np.inf)
    p = ex / np.where(live, sums, 1.0)[:, None]
    experts = np.full((t, k), -1, np.int64)
    gates = np.zeros((t, k))
    for i in np.nonzero(live)[0]:
        order = sorted((c for c in range(e) if not np.isneginf(x[i, c])), key=lambda c: (-x[i, c], c))
        for j, c in enumerate(order[:k]):
            experts[i, j] = c
            gates[i, j] = ex[i, c] if renorm else p[i, c]
    if renorm:
        total = gates.sum(1, keepdims=True)
        gates = gates / np.where(total > 0, total, 1.0)
    counts = np.bincount(experts[experts >= 0], minlength=e).astype(np.int64)
    starts = np.concatenate([[0], np.cumsum(counts)])
    slots = np.zeros((t, k), np.int64)
    at, behind = starts[:-1].copy(), int(starts[-1])
    for i in range(t):
        for j in range(k):
            c = experts[i, j]
            if c >= 0:
                slots[i, j] = at[c]
                at[c] += 1
            else:
                slots[i, j] = ~behind
                behind += 1
    offsets = np.concatenate([starts[:-1], [t * k]]).astype(np.int64)
    n = int(live.sum())
    losses = np.zeros(2)
    if n:
        losses[0] = e * (counts / (k * n) * p.sum(0) / n).sum()
        losses[1] = (np.where(live, lse, 0.0) ** 2).sum() / n
    return dict(experts=experts, gates=gates, slots=slots, lse=lse, counts=counts, offsets=offsets,
                n_tokens=n, losses=losses, p=p, live=live)


def route_bwd(r, k, d_gates, d_losses, renorm):
    """(d_logits, magnitude of its terms) for route()'s dict r."""
    p, n, live = r["p"], r["n_tokens"], r["live"]
    t, e = p.shape
    if n == 0:
        return np.zeros((t, e)), np.zeros((t, e))
    c = d_losses[0] * e * r["counts"] / (k * float(n) ** 2)
    z = np.where(live, 2.0 * d_losses[1] * np.where(live, r["lse"], 0.0) / n, 0.0)
    d = p * (c - p @ c[:, None]) + p * z[:, None]
    size = p * (np.abs(c) + p @ np.abs(c)[:, None] + np.abs(z)[:, None])
    for i in range(t):
        ch = r["experts"][i]
        sel = ch >= 0
        g, dg = r["gates"][i][sel], np.asarray(d_gates[i], np.float64)[sel]
        s, a = (g * dg).sum(), np.abs(g * dg).sum()
        if renorm:
            d[i, ch[sel]] += g * (dg - s)
            size[i, ch[sel]] += g * (np.abs(dg) + a)
        else:
            d[i] -= p[i] * s
            d[i, ch[sel]] += g * dg
            size[i] += p[i] * a
            size[i, ch[sel]] += g * np.abs(dg)
    return d, size


def dispatch(x, slots):
    t, k = slots.shape
    xs = np.zeros((t * k, x.shape[1]))
    for j in range(k):
        on = slots[:, j] >= 0
        xs[slots[on, j]] = x[on]
    return xs


def dispatch_bwd(dxs, slots):
    """(dx, sum of |terms|)."""
    t, k = slots.shape
    dx = np.zeros((t, dxs.shape[1]))
    size = np.zeros_like(dx)
    for j in range(k):
        on = slots[:, j] >= 0
        dx[on] += dxs[slots[on, j]]
        size[on] += np.abs(dxs[slots[on, j]])
    return dx, size


def combine(ys, slots, gates, residual=None):
    """(y, sum of |terms|)."""
    t, k = slots.shape
    y = np.zeros((t, ys.shape[1])) if residual is None else np.array(residual, np.float64)
    size = np.abs(y)
    for j in range(k):
        on = slots[:, j] >= 0
        term = gates[on, j, None].astype(np.float64) * ys[slots[on, j]]
        y[on] += term
        size[on] += np.abs(term)
    return y, size


def combine_bwd(dy, ys, slots, gates):
    """(dys, d_gates, sum of |terms| of d_gates)."""
    t, k = slots.shape
    dys = np.zeros((t * k, dy.shape[1]))
    dg, size = np.zeros((t, k)), np.zeros((t, k))
    for j in range(k):
        on = slots[:, j] >= 0
        rows = slots[on, j]
        dys[rows] = gates[on, j, None].astype(np.float64) * dy[on]
        dg[on, j] = (ys[rows] * dy[on]).sum(1)
        size[on, j] = np.abs(ys[rows] * dy[on]).sum(1)
    return dys, dg, size


def clip(grads, max_norm, eps):
    """(norm, coefficient)."""
    norm = np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))
    return norm, min(1.0, max_norm / (norm + eps)) if np.isfinite(norm) else max_norm / norm
