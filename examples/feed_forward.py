"""A feed-forward sublayer trained in UFP4 and served in int8.

    python examples/feed_forward.py [--steps 20] [--tokens 2048] [--hidden 512] [--ffn 1024]

Training: layer norm, a gated UFP4 layer (both projections, the activation and the
product in one kernel), a UFP4 down projection and dropout onto the residual
stream, fitted to a fixed random map; gradients are clipped by their global norm.
Serving: the same sublayer with its weights in int8, for single tokens.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from uniform_grid_fp4_amd.feedforward import Int8FeedForward, UFP4FeedForward   # noqa: E402
from uniform_grid_fp4_amd.moe import clip_grad_norm_   # noqa: E402


def train(model, steps, tokens, hidden, lr=2e-3, seed=0):
    """Returns the loss of every step."""
    dev = next(model.parameters()).device
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    x = torch.randn((tokens, hidden), device=dev, generator=g).to(torch.bfloat16)
    mix = torch.randn((hidden, hidden), device=dev, generator=g) * hidden ** -0.5
    target = x.float() + (x.float() @ mix).tanh()
    opt = torch.optim.AdamW(model.parameters(), lr=lr, weight_decay=0.0)
    trace = []
    for _ in range(steps):
        opt.zero_grad(set_to_none=True)
        loss = ((model(x).float() - target) ** 2).mean()
        loss.backward()
        clip_grad_norm_(model.parameters(), 1.0)
        opt.step()
        trace.append(loss.detach())
    return [float(v) for v in trace]


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 20), ("tokens", 2048), ("hidden", 512), ("ffn", 1024)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--p", type=float, default=0.1)
    a = ap.parse_args()
    model = UFP4FeedForward(a.hidden, a.ffn, p=a.p, device="cuda")
    trace = train(model, a.steps, a.tokens, a.hidden)
    print("loss", " ".join(f"{v:.4f}" for v in trace), flush=True)
    served = Int8FeedForward(model)
    out = served(torch.randn((1, a.hidden), device="cuda").to(torch.bfloat16))
    print("served", tuple(out.shape), out.dtype, flush=True)


if __name__ == "__main__":
    main()
