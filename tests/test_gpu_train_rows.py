"""moe_scatter, moe_gather and moe_gates_backward against plain implementations."""
import zlib

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from combine_moe_plan_gb300 import moe  # noqa: E402
from tests.gpu_util import ensure_built  # noqa: E402

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def gen(*key):
    g = torch.Generator("cuda")
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def planned(T, H, E, k, g, P=None, router=None, T_max=None):
    pool = moe.Pool(T_max or T, H, E, P or E, k, n_sets=2)
    logits = torch.randn(T, E, generator=g, device="cuda")
    ro = ri = None
    if P:
        ro = torch.arange(E + 1, dtype=torch.int32, device="cuda")
        ro[-(P - E):] += torch.arange(1, P - E + 1, dtype=torch.int32, device="cuda")
        ri = torch.randperm(P, generator=g, device="cuda").int()
    if router is None:
        pool.plan(logits, ro, ri, buf=1)
    else:
        pool.plan_routed(logits, router, None, ro, ri, buf=1)
    return pool, pool.view(1), logits


@pytest.mark.parametrize("T,H,E,k,P", [(1, 128, 1, 1, None), (1, 7168, 256, 8, None), (96, 640, 16, 4, 18),
                                       (513, 1152, 40, 32, 44), (3000, 384, 9, 3, None)])
def test_scatter_and_gather(T, H, E, k, P):
    g = gen(T, H, E, k)
    pool, v, _ = planned(T, H, E, k, g, P, T_max=T + 3)
    n = T * k
    x = torch.randn(T, H, generator=g, device="cuda").to(BF)
    x[0, :3] = torch.tensor([float("nan"), float("inf"), -0.0], device="cuda")
    rows, gates = torch.full((n + 2, H), 7.0, dtype=BF, device="cuda"), torch.full((n + 2,), 7.0, device="cuda")
    pool.scatter(x, rows, gates, buf=1)
    slot = v["slot"][:T].long().reshape(-1)
    assert pool.check() == 0
    assert torch.equal(rows[slot].view(torch.int16), x.repeat_interleave(k, 0).view(torch.int16))
    assert torch.equal(gates[slot], v["gates"][:T].reshape(-1))
    assert (rows[n:] == 7).all() and (gates[n:] == 7).all()  # rows behind the last window
    rows2 = torch.zeros_like(rows)
    pool.scatter(x, rows2, buf=1)  # without gates
    assert torch.equal(rows2[:n].view(torch.int16), rows[:n].view(torch.int16))

    d = torch.randn(n, H, generator=g, device="cuda").to(BF)
    y = pool.gather(T, d, buf=1)
    acc = torch.zeros(T, H, device="cuda")
    for j in range(k):
        acc = acc + d[v["slot"][:T, j].long()].float()  # fp32, ascending: the same roundings
    assert torch.equal(y, acc.to(BF))
    assert pool.check() == 0


def test_gather_is_the_gradient_of_scatter():
    """<scatter(x), d> = <x, gather(d)>, with whole numbers so that both are exact."""
    T, H, E, k = 37, 256, 8, 3
    g = gen("adjoint")
    pool, _, _ = planned(T, H, E, k, g)
    x, d = (torch.randint(-4, 5, s, generator=g, device="cuda").to(BF) for s in ((T, H), (T * k, H)))
    rows, _ = pool.scatter(x, torch.empty_like(d), buf=1)
    y = pool.gather(T, d, buf=1)
    assert (rows.double() * d.double()).sum() == (x.double() * y.double()).sum()


def gates_of(x, top, router):
    """The gates of moe_plan (router None) or moe_plan_routed, in 64 bits and differentiable."""
    if router is None:
        return torch.softmax(x.gather(1, top), -1)
    s = (torch.sigmoid(x) if router.score == 1 else torch.softmax(x, -1)).gather(1, top)
    if router.renorm:
        s = s / s.sum(-1, keepdim=True)
    return s * router.scale


ROUTERS = [None] + [dict(score=s, renorm=r, scale=c) for s in ("sigmoid", "softmax") for r in (True, False)
                    for c in (1.0, 2.5)] + [dict(score="sigmoid", n_group=4, topk_group=2, group_top=2)]


@pytest.mark.parametrize("fields", ROUTERS, ids=str)
@pytest.mark.parametrize("T,E,k,parts", [(1, 8, 8, 1), (96, 256, 8, 16), (37, 40, 5, 7), (530, 1024, 32, 3),
                                         (65, 64, 6, 40), (9, 4, 1, 512)])
def test_gates_backward(T, E, k, parts, fields):
    """fp32 sums of `parts` terms, then about ten roundings of the terms' sizes."""
    if fields and fields.get("n_group") and (E // 2 < k or E // 4 < 2):
        pytest.skip("no such groups")
    router = moe.Router(**fields) if fields else None
    g = gen(T, E, k, parts, str(fields))
    pool, v, logits = planned(T, 128, E, k, g, router=router)
    n = T * k
    gp = torch.randn(n, parts, generator=g, device="cuda")
    dgates, dlogits = torch.full((T, k), 7.0, device="cuda"), torch.full((T, E), 7.0, device="cuda")
    pool.gates_backward(T, gp, dgates, dlogits, router, logits if router else None, buf=1)
    assert pool.check() == 0
    slot, top = v["slot"][:T].long(), v["topk_e"][:T].long()
    p64 = gp.double()[slot]
    want, big = p64.sum(-1), p64.abs().sum(-1)
    edg = parts * 2.0 ** -24 * big + 1e-44
    assert ((dgates.double() - want).abs() <= edg).all()
    x = logits.double().requires_grad_()
    gates = gates_of(x, top, router)
    assert torch.allclose(gates.float(), v["gates"][:T], rtol=1e-5)
    dl = torch.autograd.grad(gates, x, want)[0]
    # |d gate_i / d l_e| is at most gate_i (twice with renorm), and a logit's gradient is a sum over i; k + E
    # terms' roundings and those of exp (2^-22), each relative to the largest of them
    scale = (gates.detach() * (want.abs() + edg)).sum(-1, keepdim=True)
    rel = (k + 12) * 2.0 ** -22 + E * 2.0 ** -24
    assert ((dlogits.double() - dl).abs() <= 2 * scale * rel + 2 * (gates.detach() * edg).sum(-1, keepdim=True)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gates_backward_of_rows_without_scores(score):
    """Infinite and NaN logits: their scores are 0 or 1 and so are finite the gradients."""
    T, E, k = 6, 16, 4
    logits = torch.randn(T, E, generator=gen(score), device="cuda")
    logits[0] = float("-inf")
    logits[1, 3:] = float("-inf")
    logits[2, 5] = float("nan")
    logits[3, 7] = torch.finfo(torch.float32).min
    logits[4] = torch.finfo(torch.float32).min
    router = moe.Router(score=score)
    pool = moe.Pool(T, 128, E, E, k)
    pool.plan_routed(logits, router)
    gp = torch.ones(T * k, 2, device="cuda")
    gp[::3] = -2.0
    dgates, dlogits = pool.gates_backward(T, gp, torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda"),
                                          router, logits)
    assert pool.check() == 0
    assert dlogits.isfinite().all()
    assert (dlogits[0] == 0).all() and (dlogits[1, 3:] == 0).all() and dlogits[2, 5] == 0
    v, x = pool.view(0), logits[5:].double().requires_grad_()  # an ordinary row beside them
    dg = gp.double().sum(-1)[v["slot"][5:T].long()]
    dl = torch.autograd.grad(gates_of(x, v["topk_e"][5:T].long(), router), x, dg)[0]
    assert ((dlogits[5:].double() - dl).abs() <= dg.abs().sum() * (k + 12 + E) * 2.0 ** -22).all()


def test_gates_gradient_against_differences():
    """Moving one logit moves the gates by the gradient, the plan's own gates (64-bit softmax rounded once)."""
    T, E, k = 4, 12, 3
    g = gen("diff")
    pool, v, logits = planned(T, 128, E, k, g)
    top = v["topk_e"][:T].long()
    dg = torch.randn(T, k, generator=g, device="cuda")
    gp = torch.empty(T * k, 1, device="cuda")
    gp[v["slot"][:T].reshape(-1).long(), 0] = dg.reshape(-1)
    _, dl = pool.gates_backward(T, gp, torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda"), buf=1)
    dl, step = dl.clone(), 2.0 ** -9
    for j in range(k):
        e = top[:, j]
        loss = []
        for sign in (1, -1):
            moved = logits.clone()
            moved[torch.arange(T), e] += sign * step
            gates = torch.softmax(moved.double().gather(1, top), -1)
            loss.append((gates * dg.double()).sum(-1))
        slope = (loss[0] - loss[1]) / (2 * step)
        # third derivatives of a softmax are below 1: step^2 / 6 a term; logit steps round by 2^-24 of 4
        assert ((dl[torch.arange(T), e].double() - slope).abs() <= dg.double().abs().sum(-1) * 1e-4).all()


def test_refused_states():
    T, H, E, k = 8, 128, 8, 2
    g = gen("state")
    pool, _, logits = planned(T, H, E, k, g)
    x, rows = torch.zeros(T, H, dtype=BF, device="cuda"), torch.zeros(T * k, H, dtype=BF, device="cuda")
    gp, dgates, dlogits = (torch.zeros(*s, device="cuda") for s in ((T * k, 1), (T, k), (T, E)))
    router = moe.Router()
    for call in (lambda: pool.scatter(x, rows, buf=0), lambda: pool.gather(T, rows, buf=0),  # not planned
                 lambda: pool.scatter(x[:5], rows, buf=1),                                    # another T
                 lambda: pool.gates_backward(T, gp, dgates, dlogits, router, logits, buf=1)):  # planned without a router
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.rc == moe.MOE_ERR_STATE
    pool.plan_routed(logits, router, buf=1)
    with pytest.raises(moe.MoeError) as e:
        pool.gates_backward(T, gp, dgates, dlogits, buf=1)
    assert e.value.rc == moe.MOE_ERR_STATE


def test_empty_batch():
    pool = moe.Pool(4, 128, 4, 4, 2)
    pool.plan(torch.empty(0, 4, device="cuda"))
    x = torch.empty(0, 128, dtype=BF, device="cuda")
    pool.scatter(x, x)
    pool.gather(0, x, x)
    pool.gates_backward(0, torch.empty(0, 1, device="cuda"), torch.empty(0, 2, device="cuda"),
                        torch.empty(0, 4, device="cuda"))
    assert pool.check() == 0


def test_bad_slots_are_skipped_and_reported():
    T, H, E, k = 8, 128, 8, 2
    g = gen("slots")
    pool, v, _ = planned(T, H, E, k, g)
    v["slot"][3, 1] = T * k
    rows = torch.full((T * k, H), 7.0, dtype=BF, device="cuda")
    pool.scatter(torch.zeros(T, H, dtype=BF, device="cuda"), rows, buf=1)
    assert pool.check() == moe.DEVERR_SLOT
    pool.clear_error()
    dl = torch.full((T, E), 7.0, device="cuda")
    pool.gates_backward(T, torch.zeros(T * k, 1, device="cuda"), torch.zeros(T, k, device="cuda"), dl, buf=1)
    assert pool.check() == moe.DEVERR_SLOT
    assert (dl[3] == 7).all() and (dl[:3] == 0).all()
