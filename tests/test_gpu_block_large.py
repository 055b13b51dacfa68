"""The block operators beyond the sizes of one launch, of one turn of a kernel's
loop, or of the caches, against 64 bits.

Tolerances as in the tests of each operator at small sizes (u = 2^-24, half a
step of bf16 2^-8); each test names its own."""
import pytest
import torch

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
