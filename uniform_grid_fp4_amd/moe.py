"""Transformer-block layers around the UFP4 expert GEMMs, with autograd: RMS
norm with the residual's addition, the top-k router with its balance and z
losses, an MoE block of them with two `UFP4ExpertLinear` layers, and gradient
clipping.

The expert layers take tokens sorted by expert with device offsets.  Here the
router makes both: its slots carry tokens to expert order and back, its offsets
go to the grouped GEMMs, and nothing on the way waits for the GPU, so that a
step's launches run ahead of it (and forward passes can be captured into a HIP
graph).  That takes static shapes: the rows of padding tokens, and of choices
that do not exist where experts are masked out (-inf), are zero rows of the last
expert, which quantizes and multiplies them as any others.
"""
from __future__ import annotations

from typing import Iterable, NamedTuple, Optional

import torch

from . import block as B
from . import ufp4 as U
from .autograd import first_order
from .layers import UFP4ExpertLinear, _rows


class _NormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        n = B.ufp4_rmsnorm(x, weight, residual, eps=eps)
        ctx.save_for_backward(n.h, weight, n.rstd)
        ctx.set_materialize_grads(False)
        ctx.summed = residual is not None
        return (n.y, n.h) if ctx.summed else n.y

    @staticmethod
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        if dy is None:                               # only the stream itself was used
            return dh, dh, None, None
        dx, dw = first_order(B.ufp4_rmsnorm_bwd, _rows(dy), h, weight, rstd,
                             None if dh is None else _rows(dh))
        return dx, (dx if ctx.summed else None), dw, None


class _RouteFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, valid, renorm):
        r = B.ufp4_moe_route(logits, k, valid=valid, renorm=renorm)
        ctx.save_for_backward(logits, *r[:8])
        ctx.renorm = renorm
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(r.experts, r.slots, r.lse, r.counts, r.offsets, r.n_tokens)
        return tuple(r[:8])

    @staticmethod
    def backward(ctx, _experts, d_gates, _slots, _lse, _counts, _offsets, _n, d_losses):
        if d_gates is None and d_losses is None:
            return None, None, None, None
        logits, *saved = ctx.saved_tensors
        c = lambda t: None if t is None else t.contiguous()
        return first_order(B.ufp4_moe_route_bwd, logits, B.Routing(*saved, ctx.renorm), c(d_gates),
                           c(d_losses)), None, None, None


class _DispatchFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, slots):
        ctx.save_for_backward(slots)
        return B.ufp4_moe_dispatch(x, slots)

    @staticmethod
    def backward(ctx, dxs):
        return first_order(B.ufp4_moe_dispatch_bwd, dxs.contiguous(), *ctx.saved_tensors), None


class _CombineFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, slots, gates, residual):
        ctx.save_for_backward(ys, slots, gates)
        ctx.summed = residual is not None
        return B.ufp4_moe_combine(ys, slots, gates, residual)

    @staticmethod
    def backward(ctx, dy):
        ys, slots, gates = ctx.saved_tensors
        dys, dg = first_order(B.ufp4_moe_combine_bwd, _rows(dy), ys, slots, gates)
        return dys, None, dg, (dy if ctx.summed else None)


class RMSNorm(torch.nn.Module):
    """y = h / rms(h) * weight with h = x + residual.  forward(x) returns y;
    forward(x, residual) returns (y, h), h the new residual stream.  bf16 or
    float32 rows [..., hidden]; the weight is of that type or float32."""

    def __init__(self, hidden: int, eps: float = 1e-6, device=None, dtype=torch.bfloat16):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(hidden, device=device, dtype=dtype))
        self.eps = eps

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None):
        if residual is None:
            return _NormFn.apply(_rows(x), None, self.weight, self.eps).reshape(x.shape)
        y, h = _NormFn.apply(_rows(x), _rows(residual), self.weight, self.eps)
        return y.reshape(x.shape), h.reshape(x.shape)

    @torch.no_grad()
    def quantized(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> B.NormOut:
        """For serving: the norm's rows in E4M3 with one scale each (q, scale),
        and the residual stream h; y itself is never written."""
        return B.ufp4_rmsnorm(_rows(x), self.weight, None if residual is None else _rows(residual),
                              eps=self.eps, y=False, q8=True)


class MoERouter(torch.nn.Module):
    """Top-k choice of experts: logits = x W^T, then `ufp4_moe_route`.  Returns
    a `block.Routing` whose gates and losses (balance, z) carry gradients."""

    def __init__(self, hidden: int, n_experts: int, k: int, renorm: bool = True, device=None,
                 dtype=torch.bfloat16):
        super().__init__()
        w = torch.empty((n_experts, hidden), device=device, dtype=dtype)
        torch.nn.init.normal_(w, std=hidden ** -0.5)
        self.weight = torch.nn.Parameter(w)
        self.k, self.renorm = k, renorm

    def forward(self, x: torch.Tensor, valid: Optional[torch.Tensor] = None) -> B.Routing:
        logits = torch.nn.functional.linear(_rows(x), self.weight)
        return B.Routing(*_RouteFn.apply(logits, self.k, valid, self.renorm), self.renorm)


def dispatch(x: torch.Tensor, slots: torch.Tensor) -> torch.Tensor:
    """`ufp4_moe_dispatch` with its gradient."""
    return _DispatchFn.apply(_rows(x), slots)


def combine(ys: torch.Tensor, slots: torch.Tensor, gates: torch.Tensor,
            residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """`ufp4_moe_combine` with its gradients."""
    return _CombineFn.apply(ys, slots, gates, None if residual is None else _rows(residual))


class MoEOut(NamedTuple):
    y: torch.Tensor             # the block's output, before the residual's addition
    residual: torch.Tensor      # the residual stream y belongs to
    losses: torch.Tensor        # float32 [2]: balance, z
    counts: torch.Tensor        # int64 [experts]


class UFP4MoEBlock(torch.nn.Module):
    """A pre-norm MoE block: RMS norm of x + residual, router, dispatch, two
    `UFP4ExpertLinear` layers with a SiLU between them, combine.  `gated` ("silu" or
    "gelu") makes the first a `UFP4GatedExpertLinear`, whose kernel applies that
    activation to its gate.  x and residual are bf16 [..., hidden]; `valid` (bool,
    one per token) leaves padding tokens out.  The next block's norm adds y to the
    returned residual."""

    def __init__(self, hidden: int, ffn: int, n_experts: int, k: int, seed: int = 0, device=None,
                 grid: int = U.GRID_UNIFORM, gated: Optional[str] = None):
        super().__init__()
        self.norm = RMSNorm(hidden, device=device)
        self.router = MoERouter(hidden, n_experts, k, device=device)
        self.gated = gated is not None
        if self.gated:
            from .feedforward import UFP4GatedExpertLinear   # which imports this module
            self.up = UFP4GatedExpertLinear(n_experts, hidden, ffn, act=gated, seed=seed,
                                            grid=grid, device=device)
        else:
            self.up = UFP4ExpertLinear(n_experts, hidden, ffn, seed=seed, grid=grid,
                                       device=device)
        self.down = UFP4ExpertLinear(n_experts, ffn, hidden, seed=seed + 1, grid=grid,
                                     device=device)

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                valid: Optional[torch.Tensor] = None) -> MoEOut:
        if residual is None:
            y, h = self.norm(x), x
        else:
            y, h = self.norm(x, residual)
        r = self.router(y, None if valid is None else valid.reshape(-1))
        xs = dispatch(y, r.slots)
        up = self.up(xs, r.offsets)
        ys = self.down(up if self.gated else torch.nn.functional.silu(up), r.offsets)
        out = combine(ys, r.slots, r.gates)
        return MoEOut(out.reshape(x.shape), h, r.losses, r.counts)


def clip_grad_norm_(parameters: Iterable[torch.Tensor], max_norm: float,
                    eps: float = 1e-6) -> torch.Tensor:
    """Scale the parameters' gradients in place so that their global norm is at
    most max_norm; returns the norm before it (a float32 scalar on the
    parameters' device; zero if none of them has a gradient).  A parameter that
    is listed twice, as a tied weight may be, counts and is scaled once."""
    params = [parameters] if isinstance(parameters, torch.Tensor) else list(parameters)
    grads = list({id(p.grad): p.grad for p in params if p.grad is not None}.values())
    if not grads:
        return torch.zeros((), device=params[0].device if params else None)
    return B.ufp4_clip_grads(grads, max_norm, eps=eps)
