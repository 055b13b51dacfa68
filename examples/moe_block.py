"""Two MoE blocks trained and then served with the UFP4 framework.

    python examples/moe_block.py [--steps 20] [--tokens 2048] [--hidden 512] ...

Training: each block is RMS norm (+ residual), router, dispatch, UFP4 expert
layers, combine; the loss is a regression onto a fixed random target plus the
balance and z losses; gradients are clipped by their global norm.  Part of
every batch is padding.  Serving: single tokens through the same blocks, and
the last norm's E4M3 rows into an 8-bit projection.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from uniform_grid_fp4_amd.moe import RMSNorm, UFP4MoEBlock, clip_grad_norm_   # noqa: E402


class Model(torch.nn.Module):
    def __init__(self, hidden, ffn, experts, k, layers, device):
        super().__init__()
        self.blocks = torch.nn.ModuleList(
            UFP4MoEBlock(hidden, ffn, experts, k, seed=2 * i, device=device)
            for i in range(layers))
        self.norm = RMSNorm(hidden, device=device)

    def stream(self, x, valid=None):
        """(last block's output, residual stream, summed losses)."""
        y, residual, losses = x, None, 0.0
        for block in self.blocks:
            y, residual, more, _ = block(y, residual, valid)
            losses = losses + more
        return y, residual, losses

    def forward(self, x, valid=None):
        y, residual, losses = self.stream(x, valid)
        return self.norm(y, residual)[0], losses


def train(model, steps, tokens, hidden, max_norm=1.0, lr=2e-3, seed=0):
    """Returns the regression loss of every step."""
    dev = next(model.parameters()).device
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    x = torch.randn((tokens, hidden), device=dev, generator=g).to(torch.bfloat16)
    mix = torch.randn((hidden, hidden), device=dev, generator=g) * hidden ** -0.5
    target = x.float() @ mix
    valid = torch.arange(tokens, device=dev) < tokens - tokens // 8
    opt = torch.optim.AdamW(model.parameters(), lr=lr, weight_decay=0.0)
    trace = []
    for _ in range(steps):
        opt.zero_grad(set_to_none=True)
        y, losses = model(x, valid)
        fit = ((y.float() - target)[valid] ** 2).mean()
        (fit + 0.01 * losses[0] + 0.001 * losses[1]).backward()
        clip_grad_norm_(model.parameters(), max_norm)
        opt.step()
        trace.append(fit.detach())
    return [float(v) for v in trace]


@torch.no_grad()
def serve(model, x):
    """One pass over a few tokens; the last norm in E4M3, then an 8-bit
    projection with its rows' and the weight's scales."""
    hidden = x.shape[-1]
    y, residual, _ = model.stream(x)
    n = model.norm.quantized(y, residual)
    w = torch.eye(hidden, device=x.device)
    w_scale = w.abs().amax(1) / 448.0
    w8 = (w / w_scale[:, None]).to(torch.float8_e4m3fn)
    return torch._scaled_mm(n.q, w8.t(), scale_a=n.scale[:, None], scale_b=w_scale[None, :],
                            out_dtype=torch.bfloat16)


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 20), ("tokens", 2048), ("hidden", 512), ("ffn", 512),
                        ("experts", 16), ("k", 2), ("layers", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    model = Model(a.hidden, a.ffn, a.experts, a.k, a.layers, "cuda")
    trace = train(model, a.steps, a.tokens, a.hidden)
    print("loss", " ".join(f"{v:.4f}" for v in trace), flush=True)
    out = serve(model, torch.randn((1, a.hidden), device="cuda").to(torch.bfloat16))
    print("served", tuple(out.shape), out.dtype, flush=True)


if __name__ == "__main__":
    main()
