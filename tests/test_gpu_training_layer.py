"""layer.TrainingLayer: forward and backward together against the layer in 64 bits,
its gradients against differences, several batches in flight, captured and replayed."""
import zlib

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from combine_moe_plan_gb300 import layer, moe  # noqa: E402
from tests.gpu_util import ensure_built  # noqa: E402

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def gen(*key):
    g = torch.Generator("cuda")
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


class Problem:
    def __init__(self, T, H, I, E, k, router=None, P=None, T_max=None, n_sets=1, seed=0):
        g = gen(T, H, I, E, k, seed)
        P = P or E
        self.T, self.H, self.I, self.E, self.k, self.P = T, H, I, E, k, P
        self.w13 = (torch.randn(P, 2 * I, H, generator=g, device="cuda") * 1.5 * H ** -0.5).to(BF)
        self.w2 = (torch.randn(P, H, I, generator=g, device="cuda") * I ** -0.5).to(BF)
        self.x = torch.randn(T, H, generator=g, device="cuda").to(BF)
        self.dy = torch.randn(T, H, generator=g, device="cuda").to(BF)
        self.logits = torch.randn(T, E, generator=g, device="cuda")
        self.router = router
        ro = ri = None
        if P > E:  # the last experts have two replicas
            ro = torch.arange(E + 1, dtype=torch.int32, device="cuda")
            ro[-(P - E):] += torch.arange(1, P - E + 1, dtype=torch.int32, device="cuda")
            ri = torch.randperm(P, generator=g, device="cuda").int()
        self.layer = layer.TrainingLayer(self.w13, self.w2, T_max or T, E, k, router, rep_off=ro, rep_ids=ri, n_sets=n_sets)

    def grads(self, dtype=torch.float32):
        return (torch.empty(self.P, 2 * self.I, self.H, dtype=dtype, device="cuda"),
                torch.empty(self.P, self.H, self.I, dtype=dtype, device="cuda"))

    def forward64(self, x, logits, w13, w2, top, phys):
        """The layer's y, differentiable, for the chosen experts."""
        if self.router is None:
            gates = torch.softmax(logits.gather(1, top), -1)
        else:
            s = (torch.sigmoid(logits) if self.router.score == 1 else torch.softmax(logits, -1)).gather(1, top)
            gates = (s / s.sum(-1, keepdim=True) if self.router.renorm else s) * self.router.scale
        y = torch.zeros(self.T, self.H, dtype=x.dtype, device=x.device)
        for p in range(self.P):
            t, j = (phys == p).nonzero(as_tuple=True)
            if t.numel():
                gu = x[t] @ w13[p].T
                h = torch.nn.functional.silu(gu[:, :self.I]) * gu[:, self.I:]
                y = y.index_add(0, t, gates[t, j, None] * (h @ w2[p].T))
        return y

    def reference(self):
        v = self.layer.views[0]
        top, phys = v["topk_e"][:self.T].long(), v["phys"][:self.T].long()
        leaves = [t.double().requires_grad_() for t in (self.x, self.logits, self.w13, self.w2)]
        y = self.forward64(*leaves, top, phys)
        return y.detach(), torch.autograd.grad(y, leaves, self.dy.double())


def close(got, want, rms_share):
    """Root mean square of the difference against that of the values."""
    far = (got.double() - want).square().mean().sqrt() / want.square().mean().sqrt().clamp_min(1e-30)
    assert far <= rms_share, float(far)


# Rounding of bf16 steps in a row (x rows are exact; h, out, dout exact, hg, dgu, dx rows, y) is 2^-8 at most
# each and independent: 3 of them in a chain leave a root mean square below 2^-8.  The codes of g and u are off by
# at most 2^-4 of the value (uniform: 2^-4 / sqrt 3 root mean square, and half of it on average over a binade),
# and reach the gradients through two factors of order one: 2 * 2^-4 / sqrt 3 = 0.073 bounds them.
FORWARD, BACKWARD = 2.0 ** -7, 0.073


@pytest.mark.parametrize("T,H,I,E,k,P,fields", [
    (64, 256, 128, 8, 2, None, None), (1, 256, 384, 4, 3, None, None), (300, 384, 256, 16, 4, 18, None),
    (130, 256, 256, 16, 4, None, dict(score="sigmoid", n_group=4, topk_group=2, group_top=2, scale=2.5)),
    (700, 128, 384, 8, 3, None, dict(score="softmax", renorm=False))], ids=str)
def test_layer_against_64_bits(T, H, I, E, k, P, fields):
    p = Problem(T, H, I, E, k, moe.Router(**fields) if fields else None, P)
    y = p.layer.forward(p.x, p.logits)
    dw13, dw2 = p.grads()
    dx, dlogits = p.layer.backward(p.dy, dw13, dw2)
    assert p.layer.check() == 0
    want, (rx, rl, r13, r2) = p.reference()
    close(y, want, FORWARD)
    for got, ref in ((dx, rx), (dlogits, rl), (dw13, r13), (dw2, r2)):
        close(got, ref, BACKWARD)
    b13, b2 = p.grads(BF)
    p.layer.forward(p.x, p.logits)
    dx2, dl2 = p.layer.backward(p.dy, b13, b2)
    assert torch.equal(dx, dx2) and torch.equal(dlogits, dl2)
    assert torch.equal(b13, dw13.to(BF)) and torch.equal(b2, dw2.to(BF))


def test_gradients_against_differences():
    """The layer's own y, moved along its gradients: the slope of <y, dy> is the
    gradient's length.  y is bf16 (2^-8 of each value, independent), so the
    difference of two sums over T H values is good to 2^-8 sqrt(2 T H) rms(y dy)."""
    p = Problem(256, 256, 256, 4, 2)
    p.layer.forward(p.x, p.logits)
    dw13, dw2 = p.grads()
    dx, _ = p.layer.backward(p.dy, dw13, dw2)

    def loss(x, w13, w2):
        lay = layer.TrainingLayer(w13, w2, p.T, p.E, p.k)
        y = lay.forward(x, p.logits)
        prod = y.double() * p.dy.double()
        return prod.sum().item(), prod.square().mean().sqrt().item()

    for name, d in (("x", dx), ("w13", dw13), ("w2", dw2)):
        base = getattr(p, name)
        d = d.double()
        step = 0.05 * base.double().square().mean().sqrt() / d.square().mean().sqrt()
        ends, moved = [], []
        for sign in (1, -1):
            at = (base.double() + sign * step * d).to(BF)  # the rounded point is what is evaluated
            moved.append(at.double())
            ends.append(loss(*[at if n == name else getattr(p, n) for n in ("x", "w13", "w2")]))
        rise, predicted = ends[0][0] - ends[1][0], ((moved[0] - moved[1]) * d).sum().item()
        noise = 2.0 ** -8 * (2 * p.T * p.H) ** 0.5 * ends[0][1] * 2
        # cubic terms of a step of 5 %, and the codes' share of the gradient
        assert abs(rise - predicted) <= noise + BACKWARD * abs(predicted), (name, rise, predicted, noise)


def test_sets_in_flight_and_accumulation():
    """Two batches forward before either goes back, of different sizes, gradients added up."""
    a = Problem(96, 256, 128, 8, 2, n_sets=2)
    one13, one2 = a.grads()
    b_x, b_l, b_dy = a.x[:40] * 2, a.logits[40:80].contiguous(), a.dy[:40].contiguous()
    a.layer.forward(a.x, a.logits)
    dx_a, dl_a = a.layer.backward(a.dy, one13, one2)
    a.layer.forward(b_x, b_l)
    two13, two2 = a.grads()
    dx_b, dl_b = a.layer.backward(b_dy, two13, two2)

    sum13, sum2 = torch.zeros_like(one13), torch.zeros_like(one2)
    a.layer.forward(a.x, a.logits, buf=0)
    a.layer.forward(b_x, b_l, buf=1)
    dx0, dl0 = a.layer.backward(a.dy, sum13, sum2, accumulate=True, buf=0)
    dx1, dl1 = a.layer.backward(b_dy, sum13, sum2, accumulate=True, buf=1)
    assert a.layer.check() == 0
    assert torch.equal(dx0, dx_a) and torch.equal(dl0, dl_a) and torch.equal(dx1, dx_b) and torch.equal(dl1, dl_b)
    for got, u, v in ((sum13, one13, two13), (sum2, one2, two2)):
        assert torch.equal(got, u + v)  # one rounding either way


def test_captured_and_replayed():
    p = Problem(128, 256, 128, 8, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, dx, dl = torch.empty_like(p.x), torch.empty_like(p.x), torch.empty_like(p.logits)
    dw13, dw2 = p.grads()
    with torch.cuda.stream(s):
        p.layer.forward(p.x, p.logits, y)
        p.layer.backward(p.dy, dw13, dw2, dx, dl)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        p.layer.forward(p.x, p.logits, y)
        p.layer.backward(p.dy, dw13, dw2, dx, dl)
    p.x.copy_(torch.randn(p.x.shape, generator=gen("replay"), device="cuda"))
    p.logits.copy_(torch.randn(p.logits.shape, generator=gen("replay2"), device="cuda"))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, dx, dl, dw13, dw2)]
    p.layer.forward(p.x, p.logits, y)
    p.layer.backward(p.dy, dw13, dw2, dx, dl)
    assert p.layer.check() == 0
    for u, v in zip(got, (y, dx, dl, dw13, dw2)):
        assert torch.equal(u, v)


def test_on_another_stream():
    """Every call and every new tensor on the given stream, while the current one is busy."""
    p, q = Problem(200, 256, 128, 8, 2), Problem(200, 256, 128, 8, 2)
    dw, dv = p.grads(), q.grads()
    y = p.layer.forward(p.x, p.logits)
    dx, dl = p.layer.backward(p.dy, *dw)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(20):
        busy = busy @ busy * 1e-3
    y2 = q.layer.forward(q.x, q.logits, stream=s)
    dx2, dl2 = q.layer.backward(q.dy, *dv, stream=s)
    s.synchronize()
    for a, b in zip((y, dx, dl, *dw), (y2, dx2, dl2, *dv)):
        assert torch.equal(a, b)
    assert p.layer.check() == 0 and q.layer.check() == 0


def test_two_layers_on_two_streams_at_once():
    p = [Problem(300, 384, 256, 8, 3, seed=i) for i in range(2)]
    want = []
    for q in p:
        dw = q.grads()
        y = q.layer.forward(q.x, q.logits)
        want.append((y, *q.layer.backward(q.dy, *dw), *dw))
    streams = [torch.cuda.Stream() for _ in p]
    got = [None, None]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, q in enumerate(p):
            dw = want[i][3].clone(), want[i][4].clone()
            streams[i].wait_stream(torch.cuda.current_stream())
            y = q.layer.forward(q.x, q.logits, stream=streams[i])
            got[i] = (y, *q.layer.backward(q.dy, *dw, stream=streams[i]), *dw)
    torch.cuda.synchronize()
    for i, q in enumerate(p):
        assert q.layer.check() == 0
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b)


def test_command(capsys):
    layer.main(["--train", "--tokens", "64", "--hidden", "256", "--inner", "128", "--experts", "8", "--topk", "2",
                "--groups", "4", "--steps", "2"])
    assert "backward" in capsys.readouterr().out


def test_refusals():
    p = Problem(16, 128, 128, 4, 2)
    dw13, dw2 = p.grads()
    lay = p.layer
    with pytest.raises(ValueError):
        lay.backward(p.dy, dw13, dw2)  # no forward
    lay.forward(p.x, p.logits)
    for bad in (dict(dw13=dw13[:1]), dict(dw2=dw2.double()), dict(dy=p.dy[:8]), dict(dy=p.dy.float()),
                dict(dx=p.x[:4]), dict(dlogits=p.logits.double()), dict(buf=1),
                dict(dw13=dw13.to(BF), accumulate=True)):
        with pytest.raises(ValueError):
            lay.backward(**{"dy": p.dy, "dw13": dw13, "dw2": dw2, **bad})
    lay.backward(p.dy, dw13, dw2)
    with pytest.raises(ValueError):
        lay.backward(p.dy, dw13, dw2)  # once each
    for args in ((p.x.float(), p.logits), (p.x, p.logits[:3]), (torch.cat([p.x, p.x]), torch.cat([p.logits, p.logits]))):
        with pytest.raises(ValueError):
            lay.forward(*args)
    with pytest.raises(ValueError):
        layer.TrainingLayer(p.w13, p.w2, 4, 4, 2, bias=torch.zeros(4, device="cuda"))
    lay.forward(p.x[:0], p.logits[:0])
    dw13.fill_(1)
    dx, dl = lay.backward(p.dy[:0], dw13, dw2)
    assert dx.shape == (0, 128) and (dw13 == 0).all() and (dw2 == 0).all()
    assert lay.check() == 0
