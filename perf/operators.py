"""The operators around the expert GEMMs of a transformer block: RMS norm with
the residual's addition (and an e4m3 output with row scales), the router with
its balance loss and counts, dispatch to and combination from expert order,
and the global gradient norm with clipping.

`run` computes each in plain torch operations, or, where `own` is true, with
the calls of uniform_grid_fp4_amd.block.  Sizes follow the dense 1.5B layer
(hidden 2048, FFN 8192, 8192 tokens), the MoE 7.9B layer (64 experts, hidden
2048, FFN 1408, 16384 tokens, 6 choices) and the MoE 124B layer (hidden 6144,
FFN 2048, 65536 tokens, 8 choices) that this repository's workloads use.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
CLIP_EPS = 1e-6
D_LOSSES = (0.01, 0.001)      # the weights of the balance and the z loss


def listed():
    return [
        # one token of a serving step: residual, norm, 8-bit operand of the next projection
        dict(name="norm-token", op="norm", tokens=1, hidden=2048, type="bf16", residual=True,
             y=False, q8=True, grad=False),
        # the prefill of the MoE 124B block: the residual stream and the 8-bit operand
        dict(name="norm-q8-prefill", op="norm", tokens=32768, hidden=6144, type="bf16",
             residual=True, y=True, q8=True, grad=False),
        # one norm of the dense 1.5B training step, forward and backward
        dict(name="norm-train-dense", op="norm", tokens=8192, hidden=2048, type="bf16",
             residual=True, y=True, q8=False, grad=True),
        # odd sizes in FP32: rows that no vector load fits
        dict(name="norm-train-odd-fp32", op="norm", tokens=4099, hidden=1411, type="fp32",
             residual=False, y=True, q8=False, grad=True),
        # one token's choice of experts in a serving step
        dict(name="route-token", op="route", tokens=1, experts=64, k=6, type="fp32", padded=0.0,
             renorm=True, grad=False),
        # the router of the MoE 7.9B training step, FP32 logits
        dict(name="route-train-64", op="route", tokens=16384, experts=64, k=6, type="fp32",
             padded=0.0, renorm=False, grad=True),
        # the router of the MoE 124B training step, bf16 logits, one eighth of the batch padding
        dict(name="route-train-256", op="route", tokens=65536, experts=256, k=8, type="bf16",
             padded=0.125, renorm=True, grad=True),
        # a decode batch through the experts: to expert order and back
        dict(name="exchange-decode", op="exchange", tokens=16, hidden=6144, k=8, padded=0.0,
             residual=True, grad=False),
        # the MoE 7.9B training step's token exchange, all four directions
        dict(name="exchange-train-2048", op="exchange", tokens=16384, hidden=2048, k=6,
             padded=0.0, residual=True, grad=True),
        # the MoE 124B training step's (a quarter of its tokens), part of the batch padding
        dict(name="exchange-train-6144", op="exchange", tokens=16384, hidden=6144, k=8,
             padded=0.1, residual=True, grad=True),
        # the gradients of four dense 1.5B layers, and a small odd-sized parameter in each
        dict(name="clip-dense", op="clip", layers=4, hidden=2048, ffn=8192, experts=1, extra=65,
             ratio=0.3),
        # many small tensors: latency, not bandwidth
        dict(name="clip-many-small", op="clip", layers=48, hidden=96, ffn=250, experts=1,
             extra=7, ratio=0.45),
    ]


def _between(rng, low, high):
    """A whole number spread evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _rounded(rng, n, to):
    """Mostly a multiple of `to`, at times as it is (odd sizes)."""
    return max(to, n // to * to) if rng.random() < 0.6 else n


def draw(rng):
    op = rng.choice(["norm", "route", "exchange", "clip"])
    if op == "norm":
        hidden = _rounded(rng, _between(rng, 64, 12288), 64)
        return dict(op=op, tokens=_between(rng, 1, max(1, min(65536, 200_000_000 // hidden))),
                    hidden=hidden, type=rng.choice(["bf16", "bf16", "fp32"]),
                    residual=rng.random() < 0.7, y=True, q8=rng.random() < 0.4,
                    grad=rng.random() < 0.6)
    if op == "route":
        experts = _rounded(rng, _between(rng, 4, 512), 8)
        return dict(op=op, tokens=_between(rng, 1, min(65536, 16_000_000 // experts)),
                    experts=experts, k=rng.randint(1, min(8, experts)),
                    type=rng.choice(["bf16", "fp32"]), padded=rng.choice([0.0, 0.1, 0.4]),
                    renorm=rng.random() < 0.5, grad=rng.random() < 0.7)
    if op == "exchange":
        hidden, k = _rounded(rng, _between(rng, 64, 8192), 64), rng.randint(1, 8)
        return dict(op=op, tokens=_between(rng, 1, max(1, min(65536, 500_000_000 // (hidden * k)))),
                    hidden=hidden, k=k, padded=rng.choice([0.0, 0.1, 0.4]),
                    residual=rng.random() < 0.6, grad=rng.random() < 0.7)
    hidden = _between(rng, 32, 2048)
    return dict(op=op, layers=_between(rng, 1, 4 if hidden > 512 else 32), hidden=hidden,
                ffn=_between(rng, 16, 4 * hidden), experts=rng.randint(1, 2),
                extra=_between(rng, 1, 5000), ratio=rng.choice([0.1, 0.5, 2.0]))


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1_000_003 * int(seed) + 17)
    return g


def _normal(g, shape, std, kind=torch.float32):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g).to(kind)


def _shapes(case):
    """The gradients' shapes and types, layer by layer: matrices in bf16, norm weights and one
    small parameter in FP32."""
    h, f, e, x = case["hidden"], case["ffn"], case["experts"], case["extra"]
    layer = [((h, h), "bf16")] * 4 + [((e * f, h), "bf16"), ((e * h, f), "bf16"),
                                      ((h,), "fp32"), ((h,), "fp32"), ((x,), "fp32")]
    return layer * case["layers"]


def _views(flat, shapes, kind):
    """Views of one flat bucket, one after the other as a bucket has them: odd sizes give tensors
    that start at any element."""
    sizes = [math.prod(s) for s, t in shapes if t == kind]
    return iter(flat.split(sizes))


def prepare(case, seed):
    g = _generator(seed)
    op, s = case["op"], dict(case=case)
    if op == "norm":
        t, h, kind = case["tokens"], case["hidden"], TYPES[case["type"]]
        # activations with a few outlier channels, as the quantizer's inputs here
        loud = 1.0 + 49.0 * (torch.rand((h,), device=DEV, generator=g) < 0.01)
        s["x"] = (_normal(g, (t, h), 1.0) * loud).to(kind)
        s["residual"] = _normal(g, (t, h), 2.0, kind) if case["residual"] else None
        s["weight"] = (1.0 + _normal(g, (h,), 0.2)).to(kind)
        if case["grad"]:
            s["dy"] = _normal(g, (t, h), 1e-4, kind)
            s["dh"] = _normal(g, (t, h), 1e-4, kind) if case["residual"] else None
    elif op == "route":
        t, e = case["tokens"], case["experts"]
        # some experts are liked more than others, and bf16 logits tie often
        s["logits"] = (_normal(g, (t, e), 1.0) + _normal(g, (e,), 0.7)).to(TYPES[case["type"]])
        s["valid"] = None
        if case["padded"]:
            s["valid"] = torch.rand((t,), device=DEV, generator=g) >= case["padded"]
        if case["grad"]:
            s["dgates"] = _normal(g, (t, case["k"]), 1e-3)
            s["dlosses"] = torch.tensor(D_LOSSES, device=DEV)
    elif op == "exchange":
        t, h, k = case["tokens"], case["hidden"], case["k"]
        # rows in a random expert order; padding tokens have no row of their own: their k choices
        # hold the last rows, as ~row
        routed = torch.rand((t, 1), device=DEV, generator=g) >= case["padded"]
        key = torch.rand((t, k), device=DEV, generator=g) + (~routed)
        rows = key.reshape(-1).argsort().argsort().reshape(t, k).to(torch.int32)
        s["slots"] = torch.where(routed, rows, ~rows)
        s["gates"] = torch.rand((t, k), device=DEV, generator=g) * routed / k
        s["x"] = _normal(g, (t, h), 1.0, torch.bfloat16)
        s["ys"] = _normal(g, (t * k, h), 0.5, torch.bfloat16)
        s["residual"] = _normal(g, (t, h), 1.0, torch.bfloat16) if case["residual"] else None
        if case["grad"]:
            s["dy"] = _normal(g, (t, h), 1e-4, torch.bfloat16)
            s["dxs"] = _normal(g, (t * k, h), 1e-4, torch.bfloat16)
    else:
        shapes = _shapes(case)
        total = {k: sum(math.prod(sh) for sh, t in shapes if t == k) for k in TYPES}
        flat = {k: _normal(g, (n,), 1e-3, TYPES[k]) for k, n in total.items()}
        s["buckets"] = {k: torch.zeros_like(v) for k, v in flat.items()}
        src = {k: _views(flat[k], shapes, k) for k in TYPES}
        dst = {k: _views(s["buckets"][k], shapes, k) for k in TYPES}
        s["grads"] = [next(src[t]).view(sh) for sh, t in shapes]
        s["out"] = [next(dst[t]).view(sh) for sh, t in shapes]
        s["max_norm"] = case["ratio"] * 1e-3 * math.sqrt(sum(total.values()))
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _plain_norm(s):
    case, kind = s["case"], TYPES[s["case"]["type"]]
    w = s["weight"].float()
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(kind)
    h32 = h.float()
    rstd = torch.rsqrt(h32.square().mean(1, keepdim=True) + EPS)
    y = h32 * rstd * w
    got = dict(h=h, rstd=rstd[:, 0])
    if case["y"]:
        got["y"] = y.to(kind)
    if case["q8"]:
        top = y.abs().amax(1, keepdim=True)
        got["scale"] = (top / E4M3_MAX)[:, 0]
        got["q"] = torch.where(top > 0, y * (E4M3_MAX / top), 0.0 * y).to(E4M3)
    if case["grad"]:
        dy, xhat = s["dy"].float(), h32 * rstd
        g = dy * w
        dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
        got["dx"] = (dx if s["dh"] is None else dx + s["dh"].float()).to(kind)
        got["dw"] = (dy * xhat).sum(0).to(s["weight"].dtype)
    return got


def _plain_route(s):
    case, x = s["case"], s["logits"].float()
    t, e, k = case["tokens"], case["experts"], case["k"]
    valid = s["valid"] if s["valid"] is not None else torch.ones((t,), dtype=torch.bool, device=DEV)
    n = valid.sum().clamp(min=1).float()
    order = x.sort(dim=1, descending=True, stable=True)
    top = x.amax(1)
    lse = top + (x - top[:, None]).exp().sum(1).log()
    p = (x - lse[:, None]).exp() * valid[:, None]
    chosen = order.indices[:, :k]
    gates = (order.values[:, :k] - lse[:, None]).exp()
    if case["renorm"]:
        gates = (order.values[:, :k] - top[:, None]).exp()
        gates = gates / gates.sum(1, keepdim=True)
    gates = gates * valid[:, None]
    experts = torch.where(valid[:, None], chosen, -1)
    key = torch.where(valid[:, None], chosen, e).reshape(-1)
    counts = (key[:, None] == torch.arange(e, device=DEV)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)[:-1], counts.new_full((1,), t * k)])
    rows = key.argsort(stable=True).argsort().reshape(t, k)
    slots = torch.where(valid[:, None], rows, ~rows)
    lse = torch.where(valid, lse, -math.inf)
    share = counts.float() / (k * n)
    losses = torch.stack([e * (share * p.sum(0) / n).sum(),
                          torch.where(valid, lse, 0.0).square().sum() / n])
    got = dict(experts=experts.to(torch.int32), gates=gates, slots=slots.to(torch.int32),
               counts=counts, offsets=offsets, losses=losses, lse=lse)
    if case["grad"]:
        dbal, dz = s["dlosses"][0], s["dlosses"][1]
        c = dbal * e * share / n
        dp = c + torch.where(valid, 2.0 * dz * lse / n, 0.0)[:, None]
        d = p * (c - (p * c).sum(1, keepdim=True)) + p * (dp - c)
        dg = s["dgates"]
        if case["renorm"]:
            d = d.scatter_add(1, chosen, gates * (dg - (gates * dg).sum(1, keepdim=True)))
        else:
            v = torch.zeros_like(p).scatter(1, chosen, dg)
            d = d + p * (v - (p * v).sum(1, keepdim=True))
        got["dlogits"] = d.to(s["logits"].dtype)
    return got


def _plain_exchange(s):
    case, slots = s["case"], s["slots"]
    t, h, k = case["tokens"], case["hidden"], case["k"]
    routed = (slots >= 0)[:, :, None]
    rows = torch.where(slots >= 0, slots, ~slots).long()
    xs = torch.empty((t * k, h), dtype=torch.bfloat16, device=DEV)
    xs[rows] = torch.where(routed, s["x"][:, None, :], 0.0)
    taken = torch.where(routed, s["ys"][rows], 0.0).float()
    y = (taken * s["gates"][:, :, None]).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    got = dict(xs=xs, y=y.to(torch.bfloat16))
    if case["grad"]:
        dy = s["dy"].float()[:, None, :]
        got["dys"] = torch.empty_like(xs)
        got["dys"][rows] = torch.where(routed, dy * s["gates"][:, :, None], 0.0).to(torch.bfloat16)
        got["dgates"] = (taken * dy).sum(2)
        got["dx"] = torch.where(routed, s["dxs"][rows], 0.0).float().sum(1).to(torch.bfloat16)
    return got


def _plain_clip(s):
    squares = torch.stack([g.double().square().sum() for g in s["grads"]])
    norm = squares.sum().sqrt()
    coef = (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0).float()
    [o.copy_(g.float() * coef) for g, o in zip(s["grads"], s["out"])]
    return dict(norm=norm.float(), buckets=s["buckets"])


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _own_norm(s):
    from uniform_grid_fp4_amd import block as B
    case = s["case"]
    n = B.ufp4_rmsnorm(s["x"], s["weight"], s["residual"], eps=EPS, y=case["y"], q8=case["q8"])
    got = dict(h=n.h, rstd=n.rstd)
    if case["y"]:
        got["y"] = n.y
    if case["q8"]:
        got["scale"], got["q"] = n.scale, n.q
    if case["grad"]:
        got["dx"], got["dw"] = B.ufp4_rmsnorm_bwd(s["dy"], n.h, s["weight"], n.rstd, s["dh"])
    return got


def _own_route(s):
    from uniform_grid_fp4_amd import block as B
    case = s["case"]
    r = B.ufp4_moe_route(s["logits"], case["k"], valid=s["valid"], renorm=case["renorm"])
    got = dict(experts=r.experts, gates=r.gates, slots=r.slots, counts=r.counts,
               offsets=r.offsets, losses=r.losses, lse=r.lse)
    if case["grad"]:
        got["dlogits"] = B.ufp4_moe_route_bwd(s["logits"], r, s["dgates"], s["dlosses"])
    return got


def _own_exchange(s):
    from uniform_grid_fp4_amd import block as B
    slots = s["slots"]
    got = dict(xs=B.ufp4_moe_dispatch(s["x"], slots),
               y=B.ufp4_moe_combine(s["ys"], slots, s["gates"], s["residual"]))
    if s["case"]["grad"]:
        got["dys"], got["dgates"] = B.ufp4_moe_combine_bwd(s["dy"], s["ys"], slots, s["gates"])
        got["dx"] = B.ufp4_moe_dispatch_bwd(s["dxs"], slots)
    return got


def _own_clip(s):
    from uniform_grid_fp4_amd import block as B
    norm = B.ufp4_clip_grads(s["grads"], s["max_norm"], out=s["out"], eps=CLIP_EPS)
    return dict(norm=norm, buckets=s["buckets"])


PLAIN = dict(norm=_plain_norm, route=_plain_route, exchange=_plain_exchange, clip=_plain_clip)
OWN = dict(norm=_own_norm, route=_own_route, exchange=_own_exchange, clip=_own_clip)


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op == "norm":
        t, h, size = case["tokens"], case["hidden"], SIZE[case["type"]]
        n = t * h
        b = n * size * (1 + case["y"] + 2 * case["residual"]) + 4 * t + h * size
        b += case["q8"] * (n + 4 * t)
        f = n * (5 + case["residual"] + 3 * case["q8"])
        if case["grad"]:
            b += n * size * (3 + case["residual"]) + 4 * t + 2 * h * size
            f += n * (10 + case["residual"])
        return dict(bytes=b, flops=f)
    if op == "route":
        t, e, k, size = case["tokens"], case["experts"], case["k"], SIZE[case["type"]]
        b = t * e * size + 12 * t * k + 4 * t + 16 * e + (t if case["padded"] else 0)
        f = t * e * 6
        if case["grad"]:
            b += 2 * t * e * size + 12 * t * k + 4 * t + 8 * e
            f += t * e * 8
        return dict(bytes=b, flops=f)
    if op == "exchange":
        t, h, k = case["tokens"], case["hidden"], case["k"]
        n = t * h * 2
        b = n + n * k + n * k + n * (1 + case["residual"]) + 12 * t * k
        f = 2 * t * h * k
        if case["grad"]:
            b += n * (1 + 2 * k) + n * (k + 1) + 16 * t * k
            f += 4 * t * h * k
        return dict(bytes=b, flops=f)
    shapes = _shapes(case)
    b = sum(2 * math.prod(s) * SIZE[t] for s, t in shapes)
    return dict(bytes=b, flops=sum(3 * math.prod(s) for s, _ in shapes))


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_norm(case, s):
    kind, chunk = TYPES[case["type"]], 4096
    w, parts, dw = s["weight"].double(), [], 0.0
    for i in range(0, case["tokens"], chunk):
        at = slice(i, i + chunk)
        h = s["x"][at].double()
        if s["residual"] is not None:
            h = (h + s["residual"][at].double()).to(kind).double()   # the stream's own type
        size = ((h * h).sum(1) / case["hidden"] + EPS).sqrt()
        xhat = h / size[:, None]
        y = xhat * w
        got = dict(h=h, rstd=1.0 / size)
        if case["y"]:
            got["y"] = y
        if case["q8"]:
            got["scale"] = y.abs().max(1).values / E4M3_MAX
            got["q"] = y / got["scale"].clamp(min=1e-300)[:, None]
        if case["grad"]:
            dy = s["dy"][at].double()
            inner = (dy * w * xhat).sum(1, keepdim=True) / case["hidden"]
            got["dx"] = (dy * w - xhat * inner) / size[:, None]
            if s["dh"] is not None:
                got["dx"] = got["dx"] + s["dh"][at].double()
            dw = dw + (dy * xhat).sum(0)
        parts.append(got)
    got = {name: torch.cat([p[name] for p in parts]) for name in parts[0]}
    if case["grad"]:
        got["dw"] = dw
    return got


def _exact_route(case, s):
    t, e, k = case["tokens"], case["experts"], case["k"]
    x = s["logits"].double()
    valid = torch.ones(t, device=DEV) if s["valid"] is None else s["valid"].double()
    n = max(1.0, float(valid.sum()))
    lse = torch.logsumexp(x, 1)
    p = torch.softmax(x, 1) * valid[:, None]
    left, places, picks = x.clone(), torch.arange(e, device=DEV), []
    for _ in range(k):                       # the largest left, the lowest index among equals
        is_top = left == left.max(1, keepdim=True).values
        pick = torch.where(is_top, places, e).min(1).values
        picks.append(pick)
        left[torch.arange(t, device=DEV), pick] = -math.inf
    picks = torch.stack(picks, 1)
    hot = torch.zeros((t, e), dtype=torch.float64, device=DEV).scatter_(1, picks, 1.0)
    hot = hot * valid[:, None]
    counts = hot.sum(0)
    starts = counts.cumsum(0) - counts
    row = (starts + hot.cumsum(0) - hot).gather(1, picks)
    behind = counts.sum() + ((1 - valid).cumsum(0) - (1 - valid))[:, None] * k
    behind = behind + torch.arange(k, device=DEV)
    lost = valid[:, None] == 0
    weight = p.gather(1, picks)
    total = weight.sum(1, keepdim=True) if case["renorm"] else torch.ones_like(weight[:, :1])
    gates = torch.where(lost, 0.0, weight / torch.where(lost, 1.0, total))
    got = dict(experts=torch.where(lost, -1, picks), gates=gates,
               slots=torch.where(lost, -1 - behind, row).long(), counts=counts.long(),
               offsets=torch.cat([starts, starts.new_tensor([t * k])]).long(),
               losses=torch.stack([e * (counts * p.sum(0)).sum() / (k * n * n),
                                   (valid * lse).square().sum() / n]),
               lse=torch.where(valid > 0, lse, -math.inf))
    if case["grad"]:
        # the gradient of the whole: gates . dgates + losses . dlosses, counts held
        dbal, dz = s["dlosses"].double()
        dgates = torch.where(lost, 0.0, s["dgates"].double())
        into = (dgates - (gates * dgates).sum(1, keepdim=True)) / torch.where(lost, 1.0, total) \
            if case["renorm"] else dgates
        dp = (dbal * e * counts / (k * n * n)).expand(t, e).scatter_add(1, picks, into)
        softmax = p * (dp - (p * dp).sum(1, keepdim=True))
        got["dlogits"] = softmax + p * (2 * dz * valid * lse / n)[:, None]
    return got


def _exact_exchange(case, s):
    t, h, k, grad = case["tokens"], case["hidden"], case["k"], case["grad"]
    slots = s["slots"].long()
    place = torch.where(slots < 0, -1 - slots, slots).reshape(-1)
    mine = torch.empty_like(place)
    mine[place] = torch.arange(t * k, device=DEV)          # the choice that each row belongs to
    kept = (slots.reshape(-1) >= 0)
    keep_row = kept[mine].double()[:, None]
    gate_row = s["gates"].double().reshape(-1)[mine][:, None]
    token = mine // k
    got = dict(xs=s["x"].double()[token].mul_(keep_row), y=None)
    y = torch.zeros((t, h), dtype=torch.float64, device=DEV)
    if s["residual"] is not None:
        y += s["residual"].double()
    if grad:
        dx = torch.zeros_like(y)
        got["dys"] = s["dy"].double()[token].mul_(keep_row).mul_(gate_row)
        got["dgates"] = torch.zeros((t, k), dtype=torch.float64, device=DEV)
    place = place.reshape(t, k)
    for j in range(k):
        m = kept.reshape(t, k)[:, j, None].double()
        v = s["ys"][place[:, j]].double() * m
        y += v * s["gates"][:, j, None].double()
        if grad:
            got["dgates"][:, j] = (v * s["dy"].double()).sum(1)
            dx += s["dxs"][place[:, j]].double() * m
    got["y"] = y
    if grad:
        got["dx"] = dx
    return got


def _exact_clip(case, s):
    shapes = _shapes(case)
    flat = {k: torch.cat([g.reshape(-1).double() for g, (_, t) in zip(s["grads"], shapes)
                          if t == k]) for k in TYPES}
    norm = math.sqrt(sum(float((v * v).sum()) for v in flat.values()))
    shrink = min(1.0, s["max_norm"] / (norm + CLIP_EPS))
    return dict(norm=torch.tensor(norm, dtype=torch.float64),
                buckets={k: v * shrink for k, v in flat.items()})


EXACT = dict(norm=_exact_norm, route=_exact_route, exchange=_exact_exchange, clip=_exact_clip)


def exact(case, seed):
    return EXACT[case["op"]](case, prepare(case, seed))
