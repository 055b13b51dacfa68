"""The operators of a feed-forward sublayer: layer norm with the residual's
addition, the gated product of two projections on 4-bit operands, dropout from
a counter-based generator, and the 8-bit integer product that serves them.

`run` computes each in plain torch operations, or, where `own` is true, with
the calls of uniform_grid_fp4_amd.ffn.  Sizes follow the dense 1.5B layer
(hidden 2048, FFN 8192, 8192 tokens), the MoE 7.9B layer (64 experts, hidden
2048, FFN 1408, 16384 tokens, 6 choices) and the MoE 124B layer (hidden 6144,
FFN 2048, 32 experts on a GPU, 8 choices) that this repository's workloads use.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # one token of a serving step: the residual stream and the norm
        dict(name="norm-token", op="norm", tokens=1, hidden=2048, type="bf16", residual=True,
             bias=True, grad=False),
        # one norm of the dense 1.5B training step, forward and backward
        dict(name="norm-train-dense", op="norm", tokens=8192, hidden=2048, type="bf16",
             residual=True, bias=True, grad=True),
        # odd sizes in FP32: rows that no vector load fits
        dict(name="norm-train-odd-fp32", op="norm", tokens=4099, hidden=1411, type="fp32",
             residual=False, bias=False, grad=True),
        # a small batch of odd rows, FP32: latency
        dict(name="dropout-odd-fp32", op="dropout", tokens=257, hidden=1411, type="fp32", p=0.5,
             residual=False, grad=True),
        # the end of a sublayer of the MoE 124B training step (half of its tokens): dropout onto
        # the residual stream, and its backward
        dict(name="dropout-train-6144", op="dropout", tokens=32768, hidden=6144, type="bf16",
             p=0.1, residual=True, grad=True),
        # a small odd layer: edges of tiles, few tiles
        dict(name="gated-odd", op="gated", tokens=257, hidden=1000, ffn=333, experts=1,
             act="gelu", grad=True),
        # the feed-forward layer of the dense 1.5B training step
        dict(name="gated-train-dense", op="gated", tokens=8192, hidden=2048, ffn=8192, experts=1,
             act="silu", grad=True),
        # the experts of the MoE 7.9B training step: 16384 tokens, 6 choices
        dict(name="gated-train-experts", op="gated", tokens=98304, hidden=2048, ffn=1408,
             experts=64, act="silu", grad=True),
        # one token of a serving step through the dense 1.5B feed-forward layer
        dict(name="int8-token", op="int8", tokens=1, hidden=2048, out=8192, experts=1, act="silu",
             bias=False, type="bf16"),
        # a decode batch of 16 tokens, 8 choices, over the 32 experts of the MoE 124B layer
        dict(name="int8-decode-experts", op="int8", tokens=128, hidden=6144, out=2048, experts=32,
             act="silu", bias=False, type="bf16"),
        # odd sizes in FP32, a plain projection with a bias
        dict(name="int8-odd-fp32", op="int8", tokens=1000, hidden=1411, out=565, experts=1,
             act="none", bias=True, type="fp32"),
        # the prefill of 8192 tokens through the dense 1.5B feed-forward layer
        dict(name="int8-prefill", op="int8", tokens=8192, hidden=2048, out=8192, experts=1,
             act="silu", bias=False, type="bf16"),
    ]


def _between(rng, low, high):
    """A whole number spread evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _rounded(rng, n, to):
    """Mostly a multiple of `to`, at times as it is (odd sizes)."""
    return max(to, n // to * to) if rng.random() < 0.6 else n


def draw(rng):
    op = rng.choice(["norm", "dropout", "gated", "int8"])
    kind = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("norm", "dropout"):
        hidden = _rounded(rng, _between(rng, 16, 12288), 64)
        tokens = _between(rng, 1, max(1, min(65536, 100_000_000 // hidden)))
        case = dict(op=op, tokens=tokens, hidden=hidden, type=kind,
                    residual=rng.random() < 0.7, grad=rng.random() < 0.6)
        if op == "norm":
            return dict(case, bias=rng.random() < 0.6)
        return dict(case, p=rng.choice([0.05, 0.1, 0.25, 0.5]))
    hidden, ffn = (_rounded(rng, _between(rng, 48, 8192), 64) for _ in range(2))
    experts = rng.choice([1, 1, 8, 32])
    while experts * ffn * hidden > 200_000_000:
        ffn = ffn // 2 + 1
    top = 4e11 / (4.0 * hidden * ffn)                # operations of a pass
    tokens = _between(rng, 1, max(1, min(32768, int(top))))
    if op == "gated":
        return dict(op=op, tokens=tokens, hidden=hidden, ffn=ffn, experts=experts,
                    act=rng.choice(["silu", "silu", "gelu"]), grad=rng.random() < 0.7)
    return dict(op=op, tokens=tokens, hidden=hidden, out=ffn, experts=experts,
                act=rng.choice(["none", "silu", "gelu"]), type=kind,
                bias=experts == 1 and rng.random() < 0.4)


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1_000_003 * int(seed) + 29)
    return g


def _normal(g, shape, std, kind=torch.float32):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g).to(kind)


def _activations(g, tokens, hidden, kind):
    """Rows with a few loud channels, as the inputs of this repository's quantizers."""
    loud = 1.0 + 49.0 * (torch.rand((hidden,), device=DEV, generator=g) < 0.01)
    return (_normal(g, (tokens, hidden), 1.0) * loud).to(kind)


def _four_bits(x):
    """A weight or an activation as the 4-bit GEMMs take it: nibbles of the uniform grid (sign and
    magnitude, two a byte) and one FP32 scale for 16 elements of a row, padded with zeros."""
    rows, k = x.shape
    kpad = (k + 15) // 16 * 16
    blocks = torch.nn.functional.pad(x.float(), (0, kpad - k)).reshape(rows, kpad // 16, 16)
    scales = blocks.abs().amax(2)
    level = (blocks * (7.0 / scales.clamp(min=1e-30))[:, :, None]).round().reshape(rows, kpad)
    nibble = (level.abs() + 8.0 * (level < 0)).to(torch.uint8)
    return nibble[:, 0::2] | (nibble[:, 1::2] << 4), scales


def _eight_bits(x):
    """A weight in int8 with one FP32 scale a row; rows padded with zeros to 128 bytes."""
    top = x.float().abs().amax(1)
    q = (x.float() * (127.0 / top)[:, None]).round().to(torch.int8)
    return torch.nn.functional.pad(q, (0, -x.shape[1] % 128)), top / 127.0


def _offsets(case, seed):
    """Rows of each expert, the first experts liked more; int64 offsets as the grouped GEMMs
    take them, and the largest expert's rows."""
    rng = np.random.default_rng(seed)
    like = 1.0 + rng.random(case["experts"])
    counts = rng.multinomial(case["tokens"], like / like.sum())
    return torch.from_numpy(np.concatenate([[0], counts.cumsum()])).to(DEV), int(counts.max())


def prepare(case, seed):
    g = _generator(seed)
    op, s = case["op"], dict(case=case)
    t, h = case["tokens"], case["hidden"]
    if op in ("norm", "dropout"):
        kind = TYPES[case["type"]]
        s["x"] = _activations(g, t, h, kind)
        s["residual"] = _normal(g, (t, h), 2.0, kind) if case["residual"] else None
        s["dy"] = _normal(g, (t, h), 1e-4, kind) if case["grad"] else None
        if op == "dropout":
            s["seed"], s["offset"] = (int(seed) * 0x9E3779B97F4A7C15 + 3) % 2**64, int(seed) % 1000
            return s
        s["weight"] = (1.0 + _normal(g, (h,), 0.2)).to(kind)
        s["bias"] = _normal(g, (h,), 0.1, kind) if case["bias"] else None
        s["dh"] = _normal(g, (t, h), 1e-4, kind) if case["grad"] and case["residual"] else None
        return s
    e = case["experts"]
    if e > 1:
        s["offsets"], s["most"] = _offsets(case, seed)
    if op == "gated":
        f = case["ffn"]
        s["x"] = _four_bits(_activations(g, t, h, torch.bfloat16))
        s["w"] = _four_bits(_normal(g, (e * 2 * f, h), 0.02, torch.bfloat16))
        s["dy"] = _normal(g, (t, f), 1e-4, torch.bfloat16) if case["grad"] else None
        return s
    n = case["out"] * (1 if case["act"] == "none" else 2)
    s["x"] = _activations(g, t, h, TYPES[case["type"]])
    s["w"] = _eight_bits(_normal(g, (e * n, h), 0.02, torch.bfloat16))
    s["bias"] = _normal(g, (n,), 0.5) if case["bias"] else None
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _plain_norm(s):
    kind = TYPES[s["case"]["type"]]
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(kind)
    h32, w = h.float(), s["weight"].float()
    mean = h32.mean(1, keepdim=True)
    centred = h32 - mean
    rstd = torch.rsqrt(centred.square().mean(1, keepdim=True) + EPS)
    xhat = centred * rstd
    y = xhat * w if s["bias"] is None else xhat * w + s["bias"].float()
    got = dict(h=h, y=y.to(kind), mean=mean[:, 0], rstd=rstd[:, 0])
    if s["case"]["grad"]:
        dy = s["dy"].float()
        g = dy * w
        dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        got["dx"] = (dx if s["dh"] is None else dx + s["dh"].float()).to(kind)
        got["dw"] = (dy * xhat).sum(0).to(kind)
        if s["bias"] is not None:
            got["db"] = dy.sum(0).to(kind)
    return got


def _mul_hi_lo(a, b):
    """The halves of the 64-bit products of 32-bit numbers (in int64): a constant and a tensor."""
    low = a * (b & 0xFFFF)
    high = a * (b >> 16) + (low >> 16)
    return high >> 16, ((high & 0xFFFF) << 16) | (low & 0xFFFF)


def _philox_bits(rows, cols, seed, offset):
    """16 bits for each element: Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC'11) for eight
    columns of a row at a time, counted row by row; counter words 2 and 3 are the offset."""
    groups = (cols + 7) // 8
    at = torch.arange(rows * groups, device=DEV)
    c0, c1 = at & 0xFFFFFFFF, at >> 32
    c2, c3 = torch.full_like(at, offset & 0xFFFFFFFF), torch.full_like(at, offset >> 32)
    for r in range(10):
        k0 = ((seed & 0xFFFFFFFF) + r * 0x9E3779B9) & 0xFFFFFFFF
        k1 = ((seed >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF
        (h0, l0), (h1, l1) = _mul_hi_lo(0xD2511F53, c0), _mul_hi_lo(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
    words = torch.stack([c0, c1, c2, c3], 1)
    halves = torch.stack([words & 0xFFFF, words >> 16], 2)
    return halves.reshape(rows, groups * 8)[:, :cols]


def _threshold(p):
    return int(math.floor(p * 65536.0 + 0.5))


def _plain_dropout(s):
    case, kind = s["case"], TYPES[s["case"]["type"]]
    limit = _threshold(case["p"])
    keep = _philox_bits(case["tokens"], case["hidden"], s["seed"], s["offset"]) >= limit
    up = 65536.0 / (65536 - limit)
    y = torch.where(keep, s["x"].float() * up, 0.0)
    got = dict(y=(y if s["residual"] is None else y + s["residual"].float()).to(kind))
    if case["grad"]:
        # a backward pass has no mask from the forward one: it draws it again
        keep = _philox_bits(case["tokens"], case["hidden"], s["seed"], s["offset"]) >= limit
        got["dx"] = torch.where(keep, s["dy"].float() * up, 0.0).to(kind)
    return got


def _values(q):
    """What 4-bit rows stand for."""
    codes, scales = q
    nibble = torch.stack([codes & 15, codes >> 4], 2).reshape(codes.shape[0], -1)
    level = (nibble & 7).float()
    level = torch.where(nibble > 7, -level, level)
    blocks = level.reshape(codes.shape[0], -1, 16) * (scales / 7.0)[:, :, None]
    return blocks.reshape(level.shape)


def _product(s, x, w, n):
    """x w^T, each row with its own expert's n rows of w."""
    if s["case"]["experts"] == 1:
        return x @ w.t()
    e, most, offsets = s["case"]["experts"], s["most"], s["offsets"]
    place = offsets[:-1, None] + torch.arange(most, device=DEV)
    mine = place < offsets[1:, None]
    rows = torch.where(mine, place, 0)
    y = torch.bmm(x[rows], w.reshape(e, n, -1).transpose(1, 2).contiguous())
    out = torch.empty((x.shape[0], n), dtype=y.dtype, device=DEV)
    out[place[mine]] = y[mine]
    return out


def _act(g, act):
    if act == "silu":
        return g / (1.0 + (-g).exp())
    return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))


def _act_slope(g, act):
    if act == "silu":
        p = 1.0 / (1.0 + (-g).exp())
        return p * (1.0 + g * (1.0 - p))
    return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) \
        + g * (-0.5 * g * g).exp() * (1.0 / math.sqrt(2.0 * math.pi))


def _plain_gated(s):
    case, f, kind = s["case"], s["case"]["ffn"], torch.bfloat16
    gu = _product(s, _values(s["x"]), _values(s["w"]), 2 * f)
    y = (_act(gu[:, :f], case["act"]) * gu[:, f:]).to(kind)
    if not case["grad"]:
        return dict(y=y)
    gu = gu.to(kind)                                 # what a training step keeps
    g, u, dy = gu[:, :f].float(), gu[:, f:].float(), s["dy"].float()
    dg = dy * u * _act_slope(g, case["act"])
    return dict(y=y, gu=gu, dgu=torch.cat([dg, dy * _act(g, case["act"])], 1).to(kind))


def _plain_int8(s):
    case, kind = s["case"], TYPES[s["case"]["type"]]
    x, (wq, ws) = s["x"].float(), s["w"]
    top = x.abs().amax(1, keepdim=True)
    q = (x * torch.where(top > 0, 127.0 / top, 0.0)).round()
    n = wq.shape[0] // case["experts"]
    y = _product(s, q, wq[:, :case["hidden"]].float(), n)
    if case["experts"] == 1:
        y = y * (top / 127.0) * ws
    else:
        expert = (torch.arange(case["tokens"], device=DEV)[:, None] >= s["offsets"][1:]).sum(1)
        y = y * (top / 127.0) * ws.reshape(case["experts"], n)[expert]
    if s["bias"] is not None:
        y = y + s["bias"]
    if case["act"] != "none":
        y = _act(y[:, :n // 2], case["act"]) * y[:, n // 2:]
    return y.to(kind)


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _own_norm(s):
    from uniform_grid_fp4_amd import ffn as F
    n = F.ufp4_layernorm(s["x"], s["weight"], s["bias"], s["residual"], eps=EPS)
    got = dict(h=n.h, y=n.y, mean=n.mean, rstd=n.rstd)
    if s["case"]["grad"]:
        dx, dw, db = F.ufp4_layernorm_bwd(s["dy"], n.h, s["weight"], n.mean, n.rstd, s["dh"],
                                          bias=s["bias"] is not None)
        got.update(dx=dx, dw=dw)
        if db is not None:
            got["db"] = db
    return got


def _own_dropout(s):
    from uniform_grid_fp4_amd import ffn as F
    p, seed, offset = s["case"]["p"], s["seed"], s["offset"]
    got = dict(y=F.ufp4_dropout(s["x"], p, seed, offset, residual=s["residual"]))
    if s["case"]["grad"]:
        got["dx"] = F.ufp4_dropout(s["dy"], p, seed, offset)
    return got


def _own_gated(s):
    from uniform_grid_fp4_amd import ffn as F
    from uniform_grid_fp4_amd import ufp4 as U
    case, h = s["case"], s["case"]["hidden"]
    act = F.ACT_SILU if case["act"] == "silu" else F.ACT_GELU
    xq, wq = (U.Quantized(codes, scales, codes.shape[0], h, 2 * codes.shape[1], U.GRID_UNIFORM,
                          0, 0) for codes, scales in (s["x"], s["w"]))
    out = F.ufp4_gated_gemm(xq, wq, act, keep=case["grad"], offsets=s.get("offsets"))
    if not case["grad"]:
        return dict(y=out.y)
    return dict(y=out.y, gu=out.gu, dgu=F.ufp4_gated_bwd(s["dy"], out.gu, act))


def _own_int8(s):
    from uniform_grid_fp4_amd import ffn as F
    case = s["case"]
    act = {"none": F.ACT_NONE, "silu": F.ACT_SILU, "gelu": F.ACT_GELU}[case["act"]]
    w = F.Int8Rows(*s["w"], case["hidden"])
    return F.ufp4_int8_linear(s["x"], w, bias=s["bias"], act=act, offsets=s.get("offsets"))


PLAIN = dict(norm=_plain_norm, dropout=_plain_dropout, gated=_plain_gated, int8=_plain_int8)
OWN = dict(norm=_own_norm, dropout=_own_dropout, gated=_own_gated, int8=_own_int8)


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


def work(case):
    op, t, h = case["op"], case["tokens"], case["hidden"]
    n = t * h
    if op == "norm":
        size = SIZE[case["type"]]
        vectors = 1 + case["bias"]
        b = n * size * (2 + 2 * case["residual"]) + 8 * t + vectors * h * size
        f = n * (7 + case["residual"] + case["bias"])
        if case["grad"]:
            b += n * size * (3 + case["residual"]) + 8 * t + (1 + vectors) * h * size
            f += n * (12 + case["residual"] + case["bias"])
        return dict(bytes=b, flops=f)
    if op == "dropout":
        size = SIZE[case["type"]]
        return dict(bytes=n * size * (2 + case["residual"] + 2 * case["grad"]),
                    flops=n * (2 + case["residual"] + 2 * case["grad"]))
    e = case["experts"]
    if op == "gated":
        f = case["ffn"]
        b = (n + e * 2 * f * h) * 3 // 4 + t * f * 2 + (8 * (e + 1) if e > 1 else 0)
        if case["grad"]:
            b += t * f * 2 * (2 + 2 + 1 + 2)
        return dict(bytes=b, flops=4 * t * h * f + (30 * t * f if case["grad"] else 10 * t * f))
    out, size = case["out"], SIZE[case["type"]]
    cols = out * (1 if case["act"] == "none" else 2)
    b = n * size + e * cols * (h + 4) + t * out * size + 4 * cols * case["bias"]
    return dict(bytes=b, flops=2 * t * h * cols + 3 * n)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_norm(case, s):
    kind, chunk, parts = TYPES[case["type"]], 4096, []
    w, dw, db = s["weight"].double(), 0.0, 0.0
    for i in range(0, case["tokens"], chunk):
        at = slice(i, i + chunk)
        h = s["x"][at].double()
        if s["residual"] is not None:
            h = (h + s["residual"][at].double()).to(kind).double()   # the stream's own type
        var, mean = torch.var_mean(h, dim=1, correction=0, keepdim=True)
        size = (var + EPS).sqrt()
        xhat = (h - mean) / size
        y = xhat * w + (0.0 if s["bias"] is None else s["bias"].double())
        got = dict(h=h, y=y, mean=mean[:, 0], rstd=1.0 / size[:, 0])
        if case["grad"]:
            dy = s["dy"][at].double()
            g = dy * w
            # the component of g along the ones and along xhat leaves
            along = (g * xhat).sum(1, keepdim=True) / case["hidden"]
            got["dx"] = (g - g.sum(1, keepdim=True) / case["hidden"] - along * xhat) / size
            if s["dh"] is not None:
                got["dx"] = got["dx"] + s["dh"][at].double()
            dw, db = dw + (dy * xhat).sum(0), db + dy.sum(0)
        parts.append(got)
    got = {name: torch.cat([p[name] for p in parts]) for name in parts[0]}
    if case["grad"]:
        got["dw"] = dw
        if s["bias"] is not None:
            got["db"] = db
    return got


def _kept(case, s):
    """The mask by the generator's published definition, in numpy's unsigned words."""
    rows, cols = case["tokens"], case["hidden"]
    groups = -(-cols // 8)
    u, low = np.uint64, np.uint64(0xFFFFFFFF)
    at = np.arange(rows * groups, dtype=u)
    c = [at & low, at >> u(32), np.full_like(at, s["offset"] & 0xFFFFFFFF),
         np.full_like(at, s["offset"] >> 32)]
    key = [s["seed"] & 0xFFFFFFFF, s["seed"] >> 32]
    for _ in range(10):
        a, b = u(0xD2511F53) * c[0], u(0xCD9E8D57) * c[2]
        c = [(b >> u(32)) ^ c[1] ^ u(key[0]), b & low, (a >> u(32)) ^ c[3] ^ u(key[1]), a & low]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    bits = np.empty((rows * groups, 8), dtype=np.uint16)
    for j in range(8):
        bits[:, j] = (c[j // 2] >> u(16 * (j % 2))) & u(0xFFFF)
    kept = bits.astype(np.int32) >= _threshold(case["p"])
    return torch.from_numpy(kept.reshape(rows, groups * 8)[:, :cols].copy()).to(DEV)


def _exact_dropout(case, s):
    kept, share = _kept(case, s), 1.0 - _threshold(case["p"]) / 65536.0
    y = s["x"].double().div_(share).mul_(kept)
    if s["residual"] is not None:
        y += s["residual"].double()
    got = dict(y=y)
    if case["grad"]:
        got["dx"] = s["dy"].double().div_(share).mul_(kept)
    return got


def _by_expert(case, s, x, w):
    """x w^T in 64 bits, expert by expert."""
    e = case["experts"]
    w = w.reshape(e, w.shape[0] // e, w.shape[1])
    at = [0, x.shape[0]] if e == 1 else s["offsets"].tolist()
    return torch.cat([x[a:b] @ w[i].t() for i, (a, b) in enumerate(zip(at[:-1], at[1:]))])


def _exact_act(g, act):
    return g * torch.sigmoid(g) if act == "silu" else g * torch.special.ndtr(g)


def _exact_slope(g, act):
    if act == "silu":
        p = torch.sigmoid(g)
        return p + g * p * torch.sigmoid(-g)
    return torch.special.ndtr(g) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def _numbers(q, k):
    """The numbers that 4-bit rows stand for, in 64 bits: bit 3 is the sign."""
    codes, scales = q
    table = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, 0, -1, -2, -3, -4, -5, -6, -7],
                         dtype=torch.float64, device=DEV) / 7.0
    v = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device=DEV)
    v[:, 0::2] = table[(codes % 16).long()]
    v[:, 1::2] = table[(codes // 16).long()]
    return (v * scales.double().repeat_interleave(16, 1))[:, :k]


def _exact_gated(case, s):
    f, h = case["ffn"], case["hidden"]
    gu = _by_expert(case, s, _numbers(s["x"], h), _numbers(s["w"], h))
    g, u = gu[:, :f], gu[:, f:]
    got = dict(y=_exact_act(g, case["act"]) * u)
    if case["grad"]:
        dy = s["dy"].double()
        got.update(gu=gu, dgu=torch.cat([dy * u * _exact_slope(g, case["act"]),
                                         dy * _exact_act(g, case["act"])], 1))
    return got


def _exact_int8(case, s):
    x, (wq, ws) = s["x"].double(), s["w"]
    step = x.abs().max(1, keepdim=True).values / 127.0
    q = torch.round(x / step.clamp(min=1e-300))
    # the codes are whole numbers: rows and channels scaled before the product
    w = wq[:, :case["hidden"]].double() * ws.double()[:, None]
    y = _by_expert(case, s, q * step, w)
    if s["bias"] is not None:
        y = y + s["bias"].double()
    if case["act"] != "none":
        half = y.shape[1] // 2
        y = _exact_act(y[:, :half], case["act"]) * y[:, half:]
    return y


EXACT = dict(norm=_exact_norm, dropout=_exact_dropout, gated=_exact_gated, int8=_exact_int8)


def exact(case, seed):
    return EXACT[case["op"]](case, prepare(case, seed))
