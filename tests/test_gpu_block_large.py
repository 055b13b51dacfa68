"""The block operators beyond the sizes of one launch, of one turn of a kernel's
loop, or of the caches, against 64 bits.

Tolerances as in the tests of each operator at small sizes (u = 2^-24, half a
step of bf16 2^-8); each test names its own."""
import pytest
import torch

import test_gpu_block_exchange as X
import test_gpu_block_norm as N
import test_gpu_block_route as R
from uniform_grid_fp4_amd import block as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def test_router_of_more_tokens_than_a_launch():
    """2^28 tokens and 100: the choices and the places take three launches each.
    With two experts and one choice everything has a closed form.  A row's sum
    has two terms, so c = (2 d + 41) u as for small rows, d below 16."""
    t = (1 << 28) + 100
    g = gen(1)
    x = torch.empty((t, 2), dtype=torch.bfloat16, device=DEV).normal_(0.0, 1.5, generator=g)
    valid = torch.rand((t,), device=DEV, generator=g) < 0.9
    print(f"[route] {t} x 2, k 1", flush=True)
    r = B.ufp4_moe_route(x, 1, valid=valid, renorm=False)
    torch.cuda.synchronize()
    second = x[:, 1] > x[:, 0]                           # a tie goes to the lower expert
    pick = torch.where(valid, second.to(torch.int32), -1)
    assert torch.equal(r.experts[:, 0], pick)
    n0, n1 = int((pick == 0).sum()), int((pick == 1).sum())
    assert r.counts.tolist() == [n0, n1] and r.offsets.tolist() == [0, n0, t]
    assert int(r.n_tokens) == n0 + n1
    want = torch.zeros((t,), dtype=torch.int32, device=DEV)
    for mask, start, flip in ((pick == 0, 0, False), (pick == 1, n0, False),
                              (pick < 0, n0 + n1, True)):
        place = mask.cumsum(0, dtype=torch.int32) - 1 + start
        want = torch.where(mask, ~place if flip else place, want)
    assert torch.equal(r.slots[:, 0], want)
    del want, place, mask
    c = (2 * 16 + 41) * U
    lse = torch.logaddexp(x[:, 0].double(), x[:, 1].double())
    assert float((x.double().amax(1) - x.double().amin(1)).max()) < 16
    err = (r.lse.double() - lse).abs() <= c + 4 * U * lse.abs()
    assert bool((err | ~valid).all()) and bool((r.lse[~valid] == -float("inf")).all())
    top = (x.double().amax(1) - lse).exp() * valid
    assert bool(((r.gates[:, 0].double() - top).abs() <= c * top).all())
    n = float(n0 + n1)
    p1 = ((x[:, 1].double() - lse).exp() * valid).sum()
    balance = 2.0 * (n0 * (n - float(p1)) + n1 * float(p1)) / n / n
    z = float((torch.where(valid, lse, 0.0) ** 2).sum() / n)
    # lse's own error doubles in its square; |lse| is below 16
    assert abs(float(r.losses[0]) - balance) <= (c + 16 * U) * balance
    assert abs(float(r.losses[1]) - z) <= 2 * 16 * (c + 64 * U) + 4 * U * z
    # the backward pass walks over the tokens: the last ones
    dl = torch.tensor([0.3 * n, 0.02 * n], device=DEV)
    dg = torch.rand((t, 1), device=DEV, generator=g)
    got = B.ufp4_moe_route_bwd(x, r, dg, dl)[-70000:].double()
    x, lse, valid, dg = x[-70000:].double(), lse[-70000:], valid[-70000:], dg[-70000:].double()
    p = (x - lse[:, None]).exp() * valid[:, None]
    ce = float(dl[0]) * 2.0 * r.counts.double() / (n * n)
    zt = 2.0 * float(dl[1]) / n * torch.where(valid, lse, 0.0)[:, None]
    hot = torch.nn.functional.one_hot(second[-70000:].long(), 2).double()
    gate = (p * hot).sum(1, keepdim=True)
    d = p * (ce - (p * ce).sum(1, keepdim=True) + zt - gate * dg) + hot * gate * dg
    size = p * (ce + (p * ce).sum(1, keepdim=True) + zt.abs() + gate * dg) + hot * gate * dg
    lim = 2 * c * size + 2.0 ** -8 * (d.abs() + 2 * c * size) + 1e-36
    assert bool(((got - d).abs() <= lim).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
def test_router_beyond_one_turn_of_its_loops(dtype, renorm):
    """626 workgroups, of which the scan takes 256 a turn, and more tokens than
    the backward's grid takes in one turn (32768)."""
    t = 40001
    x = R.logits_of(t, 24, dtype, 11)
    valid = torch.rand((t,), device=DEV, generator=gen(12)) < 0.85
    R.check(x, 3, valid, renorm, seed=13)


@pytest.mark.parametrize("rows,cols", [(1000, 5), (200, 17001), (9001, 121), (1100, 700)])
@pytest.mark.parametrize("dtype,wtype", [(torch.bfloat16, torch.bfloat16),
                                         (torch.bfloat16, torch.float32),
                                         (torch.float32, torch.float32)])
def test_norm_beyond_one_turn_of_its_loops(rows, cols, dtype, wtype):
    """dw of the shortest and the longest rows from several slices of rows, and
    more rows than the backward's 512 workgroups take in one turn."""
    N.test_forward_and_backward(rows, cols, dtype, wtype)


def norm_exact(h, w):
    rstd = 1.0 / (h.square().mean(1, keepdim=True) + N.EPS).sqrt()
    return h * rstd * w, rstd


@pytest.mark.parametrize("rows,cols,dtype", [(33001, 4099, torch.bfloat16),
                                             (33001, 4096, torch.bfloat16),
                                             (12000, 6147, torch.float32)])
def test_norm_with_streaming_stores(rows, cols, dtype):
    """Outputs of 256 MB and more, in rows that end inside a vector and in rows
    that do not, the residual stream in place: tolerances as at small sizes."""
    x, res, w, dy, dh = N.inputs(rows, cols, dtype, dtype, cols)
    assert x.numel() * x.element_size() >= 1 << 28
    c, half = (cols / 64 + 32) * U, N.HALF[dtype]
    h = (x.float() + res.float()).to(dtype)
    r = B.ufp4_rmsnorm(x, w, res, eps=N.EPS, q8=True, out_h=res)
    assert r.h.data_ptr() == res.data_ptr() and torch.equal(r.h, h)
    wd, dw, dws = w.double(), 0.0, 0.0
    dx, got_dw = B.ufp4_rmsnorm_bwd(dy, r.h, w, r.rstd, dh)
    for at in torch.arange(rows, device=DEV).split(4000):
        hd, g = h[at].double(), dy[at].double() * wd
        y, rstd = norm_exact(hd, wd)
        xhat = hd * rstd
        assert bool(((r.rstd[at, None].double() - rstd).abs() <= c * rstd).all())
        lim = c * y.abs() + half * (1 + c) * y.abs() + N.TINY
        assert bool(((r.y[at].double() - y).abs() <= lim).all())
        s = r.scale[at, None].double()
        lim = (2.0 ** -4 + 4 * c) * y.abs() + s * (2.0 ** -10 + 448 * 4 * c) + N.TINY
        assert bool(((r.q[at].double() * s - y).abs() <= lim).all())
        mean = (g * xhat).mean(1, keepdim=True)
        want = rstd * (g - xhat * mean) + dh[at].double()
        size = rstd * (g.abs() + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True)) \
            + dh[at].double().abs()
        lim = 4 * c * size + half * (want.abs() + 4 * c * size) + N.TINY
        assert bool(((dx[at].double() - want).abs() <= lim).all())
        dw, dws = dw + (dy[at].double() * xhat).sum(0), dws + (dy[at].double() * xhat).abs().sum(0)
    cw = (rows + cols / 64 + 32) * U
    lim = cw * dws + half * (dw.abs() + cw * dws) + N.TINY
    assert bool(((got_dw.double() - dw).abs() <= lim).all())


@pytest.mark.parametrize("t,cols,k,dtype", [(3001, 6143, 8, torch.bfloat16),
                                            (4000, 6144, 6, torch.bfloat16),
                                            (70001, 120, 16, torch.bfloat16),
                                            (2900, 2051, 12, torch.float32)])
def test_exchange_with_streaming_accesses(t, cols, k, dtype):
    """256 MB and more in expert order, a tenth of the choices missing and their
    rows NaN: tolerances as at small sizes."""
    slots, gates, x, ys, res, dy, dxs = X.make(t, cols, k, dtype, t, padded=0.1)
    assert ys.numel() * ys.element_size() >= 1 << 28
    half, on = X.HALF[dtype], slots >= 0
    lost = (~slots[~on]).long()
    ys[lost] = dxs[lost] = float("nan")
    xs = B.ufp4_moe_dispatch(x, slots)
    dx = B.ufp4_moe_dispatch_bwd(dxs, slots)
    y = B.ufp4_moe_combine(ys, slots, gates, res)
    dys, dg = B.ufp4_moe_combine_bwd(dy, ys, slots, gates)
    assert not xs[lost].any() and not dys[lost].any()
    near = lambda got, want, size, c: bool(
        ((got.double() - want).abs() <= c * size + half * (want.abs() + c * size) + 1e-37).all())
    for at in torch.arange(t, device=DEV).split(1000 if cols > 1000 else 20000):
        o, row = on[at], slots[at].clamp(min=0).long()
        take = lambda v: torch.where(o[:, :, None], v[row].double(), 0.0)
        assert torch.equal(take(xs), x[at, None].double() * o[:, :, None])
        v, g, d = take(ys), gates[at, :, None].double(), dy[at, None].double()
        assert near(y[at], (v * g).sum(1) + res[at].double(),
                    (v * g).abs().sum(1) + res[at].double().abs(), (k + 4) * U)
        assert bool(((dg[at].double() - (v * d).sum(2)).abs()
                     <= (cols / 64 + 32) * U * (v * d).abs().sum(2) + 1e-37).all())
        want = d * g * o[:, :, None]
        assert near(take(dys), want, want.abs(), U)
        v = take(dxs)
        assert near(dx[at], v.sum(1), v.abs().sum(1), (k + 4) * U)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_gradient_norm_folds_and_clipping_streams(kind):
    """520 tensors of 17 pieces of 16384 elements: 128 of them fill a launch's
    2048 workgroups, so the third launch finds no place among the 4096 partial
    sums and folds them into one, the fourth again, and some workgroups sum and
    scale two pieces.  The outputs pass 256 MB in either type."""
    n, count = 270000, 520
    pieces = -(-n // 16384)
    assert pieces == 17 and 128 * pieces > 2048 and 1 + 2 * 2048 > 4096 and count > 4 * 128
    assert count * n * 2 >= 1 << 28
    g = gen(3)
    grads = [torch.empty((n,), device=DEV).normal_(0.0, 1e-2 * (1 + (i % 7)), generator=g).to(kind)
             for i in range(count)]
    want = torch.stack([t.double().square().sum() for t in grads]).sum().sqrt()
    norm = B.ufp4_grad_norm(grads)
    assert abs(float(norm) - float(want)) <= 2 * U * float(want)
    out = [torch.empty((n,), device=DEV) for _ in grads]
    limit = 0.37 * float(want)
    assert torch.equal(B.ufp4_clip_grads(grads, limit, out=out, eps=0.0), norm)
    kept = [t.clone() for t in grads]
    B.ufp4_clip_grads(grads, limit, eps=0.0)
    half = 2.0 ** -8 if kind == torch.bfloat16 else U
    for i, (t, o, k) in enumerate(zip(grads, out, kept)):
        e = k.double() * (limit / float(want))
        assert bool(((o.double() - e).abs() <= 5 * U * e.abs() + 1e-37).all()), i
        assert bool(((t.double() - e).abs() <= (half + 4 * U) * e.abs() + 1e-37).all()), i
