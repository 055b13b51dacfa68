"""Backward passes of the layers' autograd functions, which are computed by
library calls that autograd does not see."""
from __future__ import annotations

import torch


class _FirstOnly(torch.autograd.Function):
    @staticmethod
    def forward(ctx, t):
        return t.view_as(t)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("the UFP4 layers have no second derivatives")


def first_order(call, *args, also: bool = False):
    """call(*args), a tensor or a tuple of them.  Where a backward pass is itself
    recorded (create_graph) and an argument, or with `also` what the call has
    kept, depends on what may be differentiated, the results raise when they are
    differentiated: left unrecorded, their part of a second derivative would be
    missing without a word."""
    if not torch.is_grad_enabled():
        return call(*args)
    with torch.no_grad():
        out = call(*args)
    if not (also or any(isinstance(a, torch.Tensor) and a.requires_grad for a in args)):
        return out
    refuse = lambda t: None if t is None else _FirstOnly.apply(t.detach().requires_grad_())
    return refuse(out) if isinstance(out, torch.Tensor) else tuple(map(refuse, out))
