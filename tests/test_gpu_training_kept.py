"""What layer.TrainingLayer keeps between a set's forward and its backward, and what it
does to its caller's tensors when a call is refused."""
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


def normal(*shape, scale=1.0):
    g = torch.Generator("cuda")
    g.manual_seed(zlib.crc32(repr((shape, scale)).encode()))
    return scale * torch.randn(*shape, generator=g, device="cuda")


H, I, E, K = 256, 128, 8, 2


def net(T, router=None, n_sets=1):
    return layer.TrainingLayer(normal(E, 2 * I, H, scale=H ** -0.5).to(BF), normal(E, H, I, scale=I ** -0.5).to(BF), T, E, K,
                               router, n_sets=n_sets)


def gradients():
    return torch.empty(E, 2 * I, H, device="cuda"), torch.empty(E, H, I, device="cuda")


def occupy(stream=None):
    """Some milliseconds of work in front of whatever comes next on the stream."""
    with torch.cuda.stream(stream or torch.cuda.current_stream()):
        m = torch.zeros(8192, 8192, device="cuda")
        for _ in range(6):
            m = m @ m


@pytest.mark.parametrize("inside", [False, True])
@pytest.mark.parametrize("fields", [None, dict(score="softmax")], ids=str)
def test_tensors_let_go_of_while_another_stream_has_yet_to_read_them(fields, inside):
    """The caller drops x, logits and dy after their calls; new tensors of the same sizes, made on the stream that
    they were made on, do not get their memory before the layer's stream has read it."""
    T = 4096
    router = moe.Router(**fields) if fields else None
    lay = net(T, router)
    # made and filled like the ones below, so that their memory comes from the same places
    x0, l0, dy0 = normal(T, H).to(BF), normal(T, E), normal(T, H, scale=0.5).to(BF)
    y0 = lay.forward(x0, l0)
    want13, want2 = gradients()
    dx0, dl0 = lay.backward(dy0, want13, want2)
    s = torch.cuda.Stream()
    dw13, dw2 = gradients()
    x, logits, dy = x0.clone(), l0.clone(), dy0.clone()
    torch.cuda.synchronize()
    occupy(s)
    if inside:
        with torch.cuda.stream(s):
            y = lay.forward(x, logits)
            dx, dl = lay.backward(dy, dw13, dw2)
    else:
        y = lay.forward(x, logits, stream=s)
        dx, dl = lay.backward(dy, dw13, dw2, stream=s)
    del x, logits, dy
    fresh = [torch.full(t.shape, 3.0, dtype=t.dtype, device="cuda") for t in (x0, l0, dy0) for _ in range(4)]
    s.synchronize()
    assert lay.check() == 0
    for got, want in ((y, y0), (dx, dx0), (dl, dl0), (dw13, want13), (dw2, want2)):
        assert torch.equal(got, want)
    del fresh


@pytest.mark.parametrize("fields", [None, dict(score="softmax"), dict(score="sigmoid", scale=2.5),
                                    dict(score="softmax", renorm=False)], ids=str)
def test_logits_written_over_before_the_backward(fields):
    """Two batches whose logits come in the same buffer, both forward before either goes back."""
    T = 96
    router = moe.Router(**fields) if fields else None
    lay = net(T, router, n_sets=2)
    xs, dys = [normal(T, H).to(BF), normal(T, H, scale=2).to(BF)], [normal(T, H, scale=0.5).to(BF), normal(T, H, scale=0.1).to(BF)]
    ls = [normal(T, E), normal(T, E, scale=3)]
    want = []
    for x, l, dy in zip(xs, ls, dys):
        y = lay.forward(x, l)
        dw = gradients()
        want.append((y, *lay.backward(dy, *dw), *dw))
    buffer = torch.empty(T, E, device="cuda")
    ys = []
    for b in range(2):
        buffer.copy_(ls[b])
        ys.append(lay.forward(xs[b], buffer, buf=b))
    buffer.fill_(float("nan"))
    for b in range(2):
        dw = gradients()
        got = (ys[b], *lay.backward(dys[b], *dw, buf=b), *dw)
        for u, v in zip(got, want[b]):
            assert torch.equal(u, v)
    assert lay.check() == 0


def test_a_refused_backward_adds_nothing_up():
    """An output that the last call would refuse: the gradients are as they were, and the call repeated with a
    good one adds them up once."""
    T = 40
    lay = net(T)
    x, l, dy = normal(T, H).to(BF), normal(T, E), normal(T, H, scale=0.5).to(BF)
    lay.forward(x, l)
    dw13, dw2 = (torch.full_like(t, 2.0) for t in gradients())
    odd = torch.empty(T * E + 4, device="cuda")[1:1 + T * E].view(T, E)
    with pytest.raises(ValueError):
        lay.backward(dy, dw13, dw2, dlogits=odd, accumulate=True)
    assert (dw13 == 2).all() and (dw2 == 2).all()
    lay.backward(dy, dw13, dw2, accumulate=True)
    want13, want2 = (torch.full_like(t, 2.0) for t in gradients())
    lay.forward(x, l)
    lay.backward(dy, want13, want2, accumulate=True)
    assert torch.equal(dw13, want13) and torch.equal(dw2, want2)
    assert lay.check() == 0
