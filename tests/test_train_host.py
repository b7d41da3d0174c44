"""Host-only tests of the training calls: every refusal comes before a launch
(there is no GPU here, so a call past its checks could only report MOE_ERR_CUDA,
-6), and the binding refuses tensors that the library would misread."""
import ctypes

import pytest
import torch

from combine_moe_plan_gb300 import build as moe_build
from combine_moe_plan_gb300 import moe

GOOD, ODD = ctypes.c_void_p(1 << 41), ctypes.c_void_p((1 << 41) + 4)
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
H, I, P, N = 256, 384, 4, 8


@pytest.fixture(scope="module")
def L():
    moe_build.build()
    return moe.lib()


@pytest.fixture
def pool(L):
    d = moe.Desc(64, H, 16, 16, 4, 128, 2)
    n = ctypes.c_size_t()
    assert L.moe_pool_bytes(ctypes.byref(d), ctypes.byref(n)) == 0
    h = ctypes.c_void_p()
    assert L.moe_pool_init(ctypes.byref(d), ctypes.c_void_p(1 << 40), n, ctypes.byref(h)) == 0
    yield h
    L.moe_pool_destroy(h)


def test_scatter_and_gather_check_like_dispatch(L, pool):
    f = L.moe_scatter
    assert f(None, GOOD, 8, GOOD, GOOD, 0, None) == -1
    assert f(pool, GOOD, 8, GOOD, GOOD, 2, None) == -4
    assert f(pool, GOOD, 65, GOOD, GOOD, 0, None) == -2
    assert f(pool, GOOD, -1, GOOD, GOOD, 0, None) == -2
    assert f(pool, None, 8, GOOD, GOOD, 0, None) == -1
    assert f(pool, GOOD, 8, None, GOOD, 0, None) == -1
    for bad in ((ODD, GOOD, GOOD), (GOOD, ODD, GOOD), (GOOD, GOOD, ODD)):
        assert f(pool, bad[0], 8, bad[1], bad[2], 0, None) == -3
    assert f(pool, GOOD, 8, GOOD, None, 0, None) == -9  # no plan
    g = L.moe_gather
    assert g(None, GOOD, GOOD, 8, 0, None) == -1
    assert g(pool, None, GOOD, 8, 0, None) == -1
    assert g(pool, GOOD, None, 8, 0, None) == -1
    assert g(pool, ODD, GOOD, 8, 0, None) == -3
    assert g(pool, GOOD, ODD, 8, 0, None) == -3
    assert g(pool, GOOD, GOOD, 8, 2, None) == -4
    assert g(pool, GOOD, GOOD, 65, 0, None) == -2
    assert g(pool, GOOD, GOOD, 8, 0, None) == -9


def test_gates_backward_refusals(L, pool):
    r = ctypes.byref(moe.Router())

    def f(pool=pool, router=r, logits=GOOD, gp=GOOD, parts=3, T=8, dg=GOOD, dl=GOOD, buf=0):
        return L.moe_gates_backward(pool, router, logits, gp, parts, T, dg, dl, buf, None)

    assert f(pool=None) == -1
    assert f(buf=2) == -4
    assert f(T=65) == -2
    assert f(parts=0) == -2 and f(parts=513) == -2
    assert f(router=None) == -1 and f(logits=None) == -1  # one of the pair
    for name in ("gp", "dg", "dl"):
        assert f(**{name: None}) == -1
        assert f(**{name: ODD}) == -3
    assert f(logits=ODD) == -3
    assert f(router=ctypes.byref(moe.Router(scale=0.0))) == -2
    assert f() == -9 and f(router=None, logits=None) == -9


def _weights(P=P, H=H, I=I, w13=GOOD, w2=GOOD, err=GOOD):
    return moe.DenseWeights(P, H, I, w13, w2, err)


def _call(L, name, w, rows=N, **kw):
    order = {"moe_dense_up": ("x", "offsets", rows, "h", "codes", "scales", ("stride", 8)),
             "moe_dense_down": ("h", "offsets", rows, "out"),
             "moe_dense_down_backward": ("dout", "codes", "scales", ("stride", 8), "row_gates", "offsets", rows, "dgu",
                                         "hg", "parts"),
             "moe_dense_up_backward": ("dgu", "offsets", rows, "dx"),
             "moe_dense_up_grad": ("dgu", "x", "offsets", rows, "dw", ("grad", 0)),
             "moe_dense_down_grad": ("dout", "hg", "offsets", rows, "dw", ("grad", 0))}[name]
    args = [kw.get(a, GOOD) if isinstance(a, str) else kw.get(*a) if isinstance(a, tuple) else a for a in order]
    return getattr(L, name)(None if w is None else ctypes.byref(w), *args, None)


POINTERS = {"moe_dense_up": ("x", "offsets", "h", "codes", "scales"), "moe_dense_down": ("h", "offsets", "out"),
            "moe_dense_down_backward": ("dout", "codes", "scales", "row_gates", "offsets", "dgu", "hg", "parts"),
            "moe_dense_up_backward": ("dgu", "offsets", "dx"), "moe_dense_up_grad": ("dgu", "x", "offsets", "dw"),
            "moe_dense_down_grad": ("dout", "hg", "offsets", "dw")}


@pytest.mark.parametrize("name", POINTERS)
def test_dense_refusals(L, name):
    assert _call(L, name, None) == -1
    assert _call(L, name, _weights(err=None)) == -1
    assert _call(L, name, _weights(err=ODD)) == -3
    for bad in (dict(P=0), dict(P=4097), dict(H=200), dict(H=0), dict(H=65664), dict(I=64), dict(I=130), dict(I=65664)):
        assert _call(L, name, _weights(**bad)) == -2, bad
    assert _call(L, name, _weights(), rows=-1) == -2
    assert _call(L, name, _weights(), rows=2**31 - 1) == -2
    for p in POINTERS[name]:
        assert _call(L, name, _weights(), **{p: None}) == -1, p
        assert _call(L, name, _weights(), **{p: ODD}) == -3, p


def test_dense_strides_kinds_and_weights(L):
    for name in ("moe_dense_up", "moe_dense_down_backward"):
        for stride in (0, 4, 6, 7):  # six groups, whole 16 bytes
            assert _call(L, name, _weights(), stride=stride) == -2
    for grad in (-1, 3):
        assert _call(L, "moe_dense_up_grad", _weights(), grad=grad) == -2
    assert _call(L, "moe_dense_up", _weights(w13=None)) == -1
    assert _call(L, "moe_dense_up_backward", _weights(w13=ODD)) == -3
    assert _call(L, "moe_dense_down", _weights(w2=None)) == -1
    assert _call(L, "moe_dense_down_backward", _weights(w2=None)) == -1
    # no rows: nothing to do, or an added gradient of nothing
    for name in ("moe_dense_up", "moe_dense_down", "moe_dense_down_backward", "moe_dense_up_backward"):
        assert _call(L, name, _weights(), rows=0, **{p: None for p in POINTERS[name]}) == 0
    assert _call(L, "moe_dense_up_grad", _weights(), rows=0, dgu=None, x=None, offsets=None, grad=1) == 0


# ---- the binding ----

@pytest.fixture
def experts(L, monkeypatch):
    """DenseExperts over host tensors that nothing reads."""
    monkeypatch.setattr(moe, "_on_gpu", lambda t: True)
    monkeypatch.setattr(moe, "_device", lambda: -1)  # where host tensors say they are
    monkeypatch.setattr(moe, "_stream", lambda stream: None)
    e = moe.DenseExperts.__new__(moe.DenseExperts)
    e.P, e.H, e.I = P, H, I
    e.w13, e.w2 = torch.zeros(P, 2 * I, H, dtype=BF), torch.zeros(P, H, I, dtype=BF)
    e.error_word = torch.zeros(4, dtype=torch.int32)
    e.weights = moe.DenseWeights(P, H, I, e.w13.data_ptr(), e.w2.data_ptr(), e.error_word.data_ptr())
    e._ref = ctypes.byref(e.weights)
    return e


def _tensors():
    return dict(x=torch.zeros(N, H, dtype=BF), h=torch.zeros(N, I, dtype=BF), hg=torch.zeros(N, I, dtype=BF),
                dout=torch.zeros(N, H, dtype=BF), dx=torch.zeros(N, H, dtype=BF), out=torch.zeros(N, H, dtype=BF),
                dgu=torch.zeros(N, 2 * I, dtype=BF), codes=torch.zeros(N, 2 * I, dtype=F8), scales=torch.zeros(N, 8),
                row_gates=torch.zeros(N), gate_parts=torch.zeros(N, I // 128),
                offsets=torch.zeros(P + 1, dtype=torch.int32), dw13=torch.zeros(P, 2 * I, H), dw2=torch.zeros(P, H, I))


METHODS = {"up": ("x", "offsets", "h", "codes", "scales"), "down": ("h", "offsets", "out"),
           "down_backward": ("dout", "codes", "scales", "row_gates", "offsets", "dgu", "hg", "gate_parts"),
           "up_backward": ("dgu", "offsets", "dx"), "up_grad": ("dgu", "x", "offsets", "dw13"),
           "down_grad": ("dout", "hg", "offsets", "dw2")}


@pytest.mark.parametrize("name", METHODS)
def test_binding_takes_what_it_reads(experts, name):
    t = _tensors()

    def call(**other):
        return getattr(experts, name)(*[{**t, **other}[a] for a in METHODS[name]])

    def pad(v):  # a view of the same shape that skips elements
        return torch.zeros(*v.shape[:-1], 2 * v.shape[-1], dtype=v.dtype)[..., ::2]

    with pytest.raises(moe.MoeError) as e:
        call()
    assert e.value.rc == -6  # past every check: no GPU here
    for a in METHODS[name]:
        v = t[a]
        bads = [v.to(torch.float16) if v.dtype != torch.int32 else v.long(), pad(v)]
        if a not in ("dout", "dgu", "x", "h") or METHODS[name].index(a) > 0:  # the first tensor sets the rows
            bads.append(v[:-1])
        if a != "scales" and v.dim() > 1:
            bads.append(torch.zeros(*v.shape[:-1], v.shape[-1] + 8, dtype=v.dtype))
        for bad in bads:
            with pytest.raises(ValueError):
                call(**{a: bad})


def test_binding_odds_and_ends(experts, monkeypatch):
    t = _tensors()
    with pytest.raises(ValueError):
        experts.up(t["x"], t["offsets"], t["h"], t["codes"])  # codes without scales
    with pytest.raises(ValueError):
        experts.up_grad(t["dgu"], t["x"], t["offsets"], t["dw13"].to(BF), accumulate=True)
    with pytest.raises(ValueError):
        experts.up(t["x"], t["offsets"], t["h"], rows=N + 1)  # more rows than there are
    monkeypatch.setattr(moe, "_device", lambda: 0)
    with pytest.raises(ValueError):
        experts.up(t["x"], t["offsets"], t["h"])
    for bad in (dict(), dict(w13=torch.zeros(2, 256, dtype=BF)), dict(sizes=(2, 200, 128)), dict(sizes=(2, 128, 100)),
                dict(w13=torch.zeros(2, 256, 128)), dict(w2=torch.zeros(2, 128, 128)),
                dict(w13=torch.zeros(2, 256, 128, dtype=BF), w2=torch.zeros(3, 128, 128, dtype=BF))):
        with pytest.raises(ValueError):
            moe.DenseExperts(**bad)


def test_tensors_of_another_device(monkeypatch):
    class There:
        dtype, shape, device = torch.float32, (4,), "cuda:1"

        def get_device(self):
            return 1

    here = torch.zeros(4)
    monkeypatch.setattr(moe, "_device", lambda: -1)
    moe._on_one_gpu(here, None, here)
    with pytest.raises(ValueError):
        moe._on_one_gpu(here, There())
    monkeypatch.setattr(moe, "_device", lambda: 0)
    with pytest.raises(ValueError):
        moe._on_one_gpu(here)  # a host tensor
