"""Layers of a transformer's feed-forward sublayer around the UFP4 GEMMs, with
autograd: layer norm with the residual's addition, gated linear and expert layers
whose two projections, activation and product are one kernel, dropout whose mask
is drawn again in the backward pass instead of stored, the sublayer of them, and
the int8 layers that serve what they trained.

The gated layers follow layers.py: per tensor one dual-axis quantization, bf16
outputs from the GEMMs' epilogues, only the 4-bit operands that the backward pass
needs kept, and next to them the bf16 gate and up values.
"""
from __future__ import annotations

import copy
import itertools
from typing import Optional, Union

import torch

from . import ffn as F
from . import moe as M
from . import ufp4 as U
from .autograd import first_order
from .layers import UFP4Linear, _bf16_rows, _expert_grads, _linear_grads, _recipe, _rows, \
    draw_sign_masks

ACTS = {"silu": F.ACT_SILU, "gelu": F.ACT_GELU}


def _same_shape(x: torch.Tensor, residual: torch.Tensor) -> None:
    """As rows, tensors of other shapes could pass for one another."""
    if residual.shape != x.shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, expected {tuple(x.shape)}")


def _act_code(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"act = {act!r}: one of {sorted(ACTS)}")
    return ACTS[act]


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------
class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, bias, eps):
        n = F.ufp4_layernorm(x, weight, bias, residual, eps=eps)
        ctx.save_for_backward(n.h, weight, n.mean, n.rstd)
        ctx.set_materialize_grads(False)
        ctx.summed, ctx.shifted = residual is not None, bias is not None
        return (n.y, n.h) if ctx.summed else n.y

    @staticmethod
    def backward(ctx, dy, dh=None):
        h, weight, mean, rstd = ctx.saved_tensors
        if dy is None:                               # only the stream itself was used
            return dh, dh, None, None, None
        dx, dw, db = first_order(F.ufp4_layernorm_bwd, _rows(dy), h, weight, mean, rstd,
                                 None if dh is None else _rows(dh), ctx.shifted)
        return dx, (dx if ctx.summed else None), dw, db, None


class LayerNorm(torch.nn.Module):
    """y = (h - mean(h)) / std(h) * weight + bias with h = x + residual.
    forward(x) returns y; forward(x, residual) returns (y, h), h the new residual
    stream.  bf16 or float32 rows [..., hidden]; weight and bias are of that type
    or float32."""

    def __init__(self, hidden: int, eps: float = 1e-5, bias: bool = True, device=None,
                 dtype=torch.bfloat16):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(hidden, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(hidden, device=device, dtype=dtype)) \
            if bias else None
        self.eps = eps

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None):
        if residual is None:
            return _LayerNormFn.apply(_rows(x), None, self.weight, self.bias,
                                      self.eps).reshape(x.shape)
        _same_shape(x, residual)
        y, h = _LayerNormFn.apply(_rows(x), _rows(residual), self.weight, self.bias, self.eps)
        return y.reshape(x.shape), h.reshape(x.shape)


# ---------------------------------------------------------------------------
# Dropout
# ---------------------------------------------------------------------------
class _DropoutFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset):
        there = isinstance(offset, torch.Tensor)
        ctx.save_for_backward(*((offset,) if there else ()))
        ctx.p, ctx.seed, ctx.offset = p, seed, None if there else offset
        ctx.summed = residual is not None
        return F.ufp4_dropout(x, p, seed, offset, residual=residual)

    @staticmethod
    def backward(ctx, dy):
        # an offset on the GPU that was changed since raises here; a recomputed call
        # gives what it saved once
        offset, = ctx.saved_tensors or (ctx.offset,)
        dx = None
        if ctx.needs_input_grad[0]:
            dx = first_order(F.ufp4_dropout, _rows(dy), ctx.p, ctx.seed, offset)
        return dx, (dy if ctx.summed else None), None, None, None


def dropout(x: torch.Tensor, p: float, seed: int, offset: Union[int, torch.Tensor] = 0,
            residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """`ufp4_dropout` with its gradients: rows [..., hidden] dropped with
    probability p, onto a residual or alone.  (seed, offset) names the mask.  An
    `offset` on the GPU must hold its value until the backward pass has run."""
    if residual is not None:
        _same_shape(x, residual)
    y = _DropoutFn.apply(_rows(x), None if residual is None else _rows(residual), p, seed, offset)
    return y.reshape(x.shape)


_drawn = itertools.count(1)


def _own_seed() -> int:
    """A seed that no other layer of the process has, from torch's and the number
    drawn so far."""
    return (torch.initial_seed() + next(_drawn) * 0x9E3779B97F4A7C15) & ((1 << 64) - 1)


# Whether autograd is running a backward pass on this thread (-1: no).
_in_backward = getattr(torch._C, "_current_graph_task_id", lambda: -1)


class Dropout(torch.nn.Module):
    """forward(x, residual=None) = residual + dropout(x); in eval mode nothing is
    dropped.  Every training call draws another mask: the k-th has offset k, or
    what `offset` holds, an int64 tensor of one element on the GPU that the caller
    advances (between the replays of a captured step, for instance).  Layers of one
    seed drop the same elements; without one a layer, and a deep copy of it, has its
    own, the same in every run that seeds torch and builds its layers in one order.
    The state dict holds seed and number of calls: who loads it goes on from there.
    `forward` takes an `offset` too (as `dropout` does), in place of the layer's.  A
    call that a backward pass runs again to recompute its activations needs one: by
    count it would draw another mask than the loss had, and is refused."""

    def __init__(self, p: float, seed: Optional[int] = None,
                 offset: Optional[torch.Tensor] = None):
        super().__init__()
        if not 0.0 <= p <= 1.0:
            raise ValueError(f"p = {p}: a probability")
        self.given = seed is not None
        self.seed = seed if self.given else _own_seed()
        self.p, self.calls, self.offset = p, 0, offset

    def __deepcopy__(self, memo):
        new = memo[id(self)] = self.__class__.__new__(self.__class__)
        own = {k: v for k, v in self.__dict__.items() if k != "offset"}
        new.__dict__.update(copy.deepcopy(own, memo))
        # the caller's tensor, which a copy of it would not follow
        new.offset = memo.get(id(self.offset), self.offset)
        if not getattr(new, "given", True):          # absent in older pickles
            new.seed = _own_seed()
        return new

    def get_extra_state(self) -> torch.Tensor:
        seed = self.seed & ((1 << 64) - 1)
        return torch.tensor([seed - (seed >> 63 << 64), self.calls], dtype=torch.int64,
                            device="cpu")

    def set_extra_state(self, state: torch.Tensor) -> None:
        seed, self.calls = state.tolist()
        self.seed = seed & ((1 << 64) - 1)

    def _load_from_state_dict(self, state_dict, prefix, metadata, strict, *more):
        # a state dict without the extra state is one from before there was any
        strict = strict and prefix + "_extra_state" in state_dict
        super()._load_from_state_dict(state_dict, prefix, metadata, strict, *more)

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                offset: Union[int, torch.Tensor, None] = None) -> torch.Tensor:
        p = self.p if self.training else 0.0
        if p == 0.0 and residual is None:
            return x
        if offset is None:
            offset = self.offset
        if offset is None:
            if p > 0.0:
                if _in_backward() != -1:
                    raise RuntimeError("a dropout that a backward pass recomputes needs an offset")
                self.calls += 1
            offset = self.calls
        return dropout(x, p, self.seed, offset, residual)


# ---------------------------------------------------------------------------
# Gated layers
# ---------------------------------------------------------------------------
class _GatedFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, n_experts, act, keep, masks, grid, seed, rht, rnd_dy):
        ctx.w_shape = w.shape
        ctx.experts = offsets is not None
        if x.shape[0] == 0:
            return x.new_empty((0, w.shape[0] // (2 * n_experts)))
        mf, md, mw = masks
        rf, rd, rw = rht
        xq, xtq = U.ufp4_rht_quantize_dual(x, (rf, mf, 0), (rw, mw, 0), grid=grid,
                                           group_offsets=offsets)
        more = dict(col_axis=U.BLOCKS_ALONG_ROWS_STACKED, n_groups=n_experts) \
            if ctx.experts else {}
        wq, wtq = U.ufp4_rht_quantize_dual(w, (rf, mf, 0), (rd, md, 0), grid=grid, **more)
        y, gu = F.ufp4_gated_gemm(xq, wq, act, keep=keep, offsets=offsets)
        ctx.q = (xtq, wtq)
        ctx.gu, ctx.act, ctx.offsets = gu, act, offsets
        ctx.masks, ctx.grid, ctx.seed, ctx.rht, ctx.rnd_dy = masks, grid, seed, rht, rnd_dy
        return y

    @staticmethod
    def backward(ctx, dy):
        # dX and dW depend on both through the gate and up values
        dx, dw = first_order(_gated_grads, ctx, dy, also=True)
        return (dx, dw) + (None,) * 9


def _gated_grads(ctx, dy):
    grads = _expert_grads if ctx.experts else _linear_grads
    if dy.shape[0] == 0:
        return grads(ctx, dy)
    if ctx.gu is None:
        raise RuntimeError("the gated layer's backward pass has run: what it kept is gone")
    # the gradient takes the place of the gate and up values
    gu, ctx.gu = ctx.gu, None
    return grads(ctx, F.ufp4_gated_bwd(_bf16_rows(dy), gu, ctx.act, out=gu))


def _gated(layer, x, offsets, n_experts):
    x = _bf16_rows(x)
    layer.sr_seed = (layer.sr_seed + 1) & ((1 << 64) - 1)
    keep = torch.is_grad_enabled() and (x.requires_grad or layer.weight.requires_grad)
    return _GatedFn.apply(x, layer.weight, offsets, n_experts, layer.act, keep, layer.masks,
                          layer.grid, layer.sr_seed, layer.rht, layer.rnd_dy)


class UFP4GatedLinear(torch.nn.Module):
    """y = act(x Wg^T) * (x Wu^T), weight [2 * ffn, in_features] in bf16 (Wg's rows,
    then Wu's); x is bf16 [..., in_features]; the output and both gradients are
    bf16.  `act` is "silu" or "gelu"; `rht` and `sr_dy` as for UFP4Linear, of the two
    projections as one product.  The gradient of the gate and up values takes their
    place, so a graph is good for one backward pass; a second one raises."""

    def __init__(self, in_features: int, ffn: int, act: str = "silu", seed: int = 0,
                 grid: int = U.GRID_UNIFORM, device=None, rht=(True, True, True),
                 sr_dy: bool = True):
        super().__init__()
        w = torch.empty((2 * ffn, in_features), device=device, dtype=torch.bfloat16)
        torch.nn.init.normal_(w, std=in_features ** -0.5)
        self.weight = torch.nn.Parameter(w)
        self.act = _act_code(act)
        self.masks = draw_sign_masks(seed)
        self.grid = grid
        self.rht, self.rnd_dy = _recipe(rht, sr_dy)
        self.sr_seed = (seed * 0x9E3779B97F4A7C15) & ((1 << 64) - 1)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        y = _gated(self, x, None, 1)
        return y.reshape(*x.shape[:-1], y.shape[-1])


class UFP4GatedExpertLinear(torch.nn.Module):
    """UFP4GatedLinear for the experts of an MoE block: tokens sorted by expert with
    device int64 offsets as UFP4ExpertLinear takes them, weights stacked [n_experts *
    2 * ffn, in_features], each expert's Wg before its Wu."""

    def __init__(self, n_experts: int, in_features: int, ffn: int, act: str = "silu",
                 seed: int = 0, grid: int = U.GRID_UNIFORM, device=None, rht=(True, True, True),
                 sr_dy: bool = True):
        super().__init__()
        w = torch.empty((n_experts * 2 * ffn, in_features), device=device, dtype=torch.bfloat16)
        torch.nn.init.normal_(w, std=in_features ** -0.5)
        self.weight = torch.nn.Parameter(w)
        self.n_experts = n_experts
        self.act = _act_code(act)
        self.masks = draw_sign_masks(seed)
        self.grid = grid
        self.rht, self.rnd_dy = _recipe(rht, sr_dy)
        self.sr_seed = (seed * 0x9E3779B97F4A7C15) & ((1 << 64) - 1)

    def forward(self, x: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
        assert offsets.dtype == torch.int64 and offsets.numel() == self.n_experts + 1
        return _gated(self, x, offsets, self.n_experts)


class UFP4FeedForward(torch.nn.Module):
    """A pre-norm feed-forward sublayer: h = x + residual, then h + dropout(down(
    gated(norm(h)))), the new residual stream.  x and residual are bf16 [...,
    hidden]; without a residual h is x.  `seed` is that of the products (0 without
    one) and of the dropout (its own without one); `offset`, of the layer or of a
    call, is the dropout's (see Dropout: captured and recomputed calls need one)."""

    def __init__(self, hidden: int, ffn: int, p: float = 0.0, act: str = "silu",
                 seed: Optional[int] = None, device=None, grid: int = U.GRID_UNIFORM,
                 offset: Optional[torch.Tensor] = None):
        super().__init__()
        self.norm = LayerNorm(hidden, device=device)
        given, seed = seed, 0 if seed is None else seed
        self.gated = UFP4GatedLinear(hidden, ffn, act=act, seed=seed, grid=grid, device=device)
        self.down = UFP4Linear(ffn, hidden, seed=seed + 1, grid=grid, device=device)
        self.drop = Dropout(p, seed=given, offset=offset)

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                offset: Union[int, torch.Tensor, None] = None) -> torch.Tensor:
        if residual is None:
            y, h = self.norm(x), x
        else:
            y, h = self.norm(x, residual)
        return self.drop(self.down(self.gated(y)), h, offset)


# ---------------------------------------------------------------------------
# Serving in int8
# ---------------------------------------------------------------------------
class Int8Linear(torch.nn.Module):
    """A trained weight in int8 with a scale for each output channel: y = x W^T (+
    bias), each token quantized on the way.  With an `act` ("silu", "gelu") the
    weight has gate rows, then up rows, and y = act(gate) * up.  n_experts > 1: the
    weights of as many experts, stacked, and forward takes their offsets.  For
    serving: no gradients."""

    def __init__(self, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 act: Optional[str] = None, n_experts: int = 1):
        super().__init__()
        self.act = F.ACT_NONE if act is None else _act_code(act)
        F._rows_per_group(weight.shape[0], n_experts, 1 if act is None else 2)
        self.n_experts = n_experts
        w = F.ufp4_int8_quantize(_rows(weight.detach()))
        self.register_buffer("q", w.q)
        self.register_buffer("scale", w.scale)
        self.register_buffer("bias", None if bias is None else bias.detach().float().contiguous())
        self.in_features = w.k

    def _apply(self, fn, *more):
        """Moves go through; a cast of the model's floating-point numbers leaves the
        scales and the bias, which are FP32 whatever the activations are."""
        had = {n: t for n, t in self.named_buffers(recurse=False) if t.is_floating_point()}
        super()._apply(fn, *more)
        for n, t in had.items():
            if self._buffers[n].dtype != t.dtype:
                self._buffers[n] = t.to(self._buffers[n].device)
        return self

    @torch.no_grad()
    def forward(self, x: torch.Tensor, offsets: Optional[torch.Tensor] = None) -> torch.Tensor:
        if (offsets is None) != (self.n_experts == 1) or \
                (offsets is not None and offsets.numel() != self.n_experts + 1):
            raise ValueError(f"offsets of {self.n_experts} experts")
        y = F.ufp4_int8_linear(_rows(x), F.Int8Rows(self.q, self.scale, self.in_features),
                               bias=self.bias, act=self.act, offsets=offsets)
        return y.reshape(*x.shape[:-1], y.shape[-1])


def _act_name(code: int) -> str:
    return next(name for name, c in ACTS.items() if c == code)


class Int8FeedForward(torch.nn.Module):
    """What serves a trained UFP4FeedForward: its norm (the same module), and its
    products in int8 (of the weights as they are now)."""

    def __init__(self, trained: UFP4FeedForward):
        super().__init__()
        self.norm = trained.norm
        self.gated = Int8Linear(trained.gated.weight, act=_act_name(trained.gated.act))
        self.down = Int8Linear(trained.down.weight)

    @torch.no_grad()
    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        if residual is None:
            y, h = self.norm(x), x
        else:
            y, h = self.norm(x, residual)
        return dropout(self.down(self.gated(y)), 0.0, 0, residual=h)


class Int8MoEBlock(torch.nn.Module):
    """What serves a trained gated `moe.UFP4MoEBlock`: its norm and router (the same
    modules), and its experts' products in int8 (of the weights as they are now)."""

    def __init__(self, trained: "M.UFP4MoEBlock"):
        super().__init__()
        if not isinstance(trained.up, UFP4GatedExpertLinear):
            raise TypeError("Int8MoEBlock serves a block with gated experts")
        self.norm, self.router = trained.norm, trained.router
        e = trained.up.n_experts
        self.up = Int8Linear(trained.up.weight, act=_act_name(trained.up.act), n_experts=e)
        self.down = Int8Linear(trained.down.weight, n_experts=e)

    @torch.no_grad()
    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                valid: Optional[torch.Tensor] = None) -> "M.MoEOut":
        if residual is None:
            y, h = self.norm(x), x
        else:
            y, h = self.norm(x, residual)
        r = self.router(y, None if valid is None else valid.reshape(-1))
        at = r.offsets if self.up.n_experts > 1 else None
        ys = self.down(self.up(M.dispatch(y, r.slots), at), at)
        out = M.combine(ys, r.slots, r.gates)
        return M.MoEOut(out.reshape(x.shape), h, r.losses, r.counts)
