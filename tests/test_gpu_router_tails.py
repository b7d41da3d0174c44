"""moe_gates_backward where all chosen scores of a token are tiny but not zero: the
renormalised gates, and their gradients, are of ordinary size."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from combine_moe_plan_gb300 import moe  # noqa: E402
from tests.gpu_util import ensure_built  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("lowest", [-60.0, -87.0, -88.5])
def test_scores_near_the_smallest(score, lowest):
    """fp32 against 64 bits.  A score is off by a few 2^-22 of itself and by up to 2^-148 (two roundings of numbers
    below the normal ones); a gate's share r = s / S of the gradient by that and k roundings of the sum, twice."""
    T, E, k = 7, 16, 4
    g = torch.Generator("cuda")
    g.manual_seed(int(-lowest))
    logits = torch.full((T, E), -200.0, device="cuda")
    tiny = lowest + torch.rand(T, 6, generator=g, device="cuda")
    bias = None
    if score == "sigmoid":
        logits[:, 5:11] = tiny  # the others' scores are 0
    else:
        logits = torch.randn(T, E, generator=g, device="cuda")
        logits[:, 5:11] = logits.amax(-1, keepdim=True) + tiny
        bias = torch.zeros(E, device="cuda")
        bias[5:11] = 2.0  # chosen for the bias
    router = moe.Router(score=score, renorm=True, scale=2.5)
    pool = moe.Pool(T, 128, E, E, k)
    pool.plan_routed(logits, router, bias)
    gp = 9 * torch.randn(T * k, 3, generator=g, device="cuda")
    dgates, dlogits = pool.gates_backward(T, gp, torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda"),
                                          router, logits)
    assert pool.check() == 0
    v = pool.view(0)
    slot, top = v["slot"][:T].long(), v["topk_e"][:T].long()
    assert ((top >= 5) & (top < 11)).all()
    dg = gp.double()[slot].sum(-1)
    x = logits.double().requires_grad_()
    s = (torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, -1)).gather(1, top)
    gates = 2.5 * s / s.sum(-1, keepdim=True)
    want = torch.autograd.grad(gates, x, dg)[0]
    rel = (k + 12) * 2.0 ** -22 + E * 2.0 ** -24 + 2.0 ** -148 / s.detach().min()
    scale = (gates.detach() * gp.double()[slot].abs().sum(-1)).sum(-1, keepdim=True)
    assert want.abs().max() > 1
    assert ((dlogits.double() - want).abs() <= 2 * scale * rel).all()
