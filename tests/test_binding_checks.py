"""The Python entry points of the expert layer refuse tensors that the library
would misread or read past the end of: type, shape, strides and device.

There is no GPU here: host tensors stand for device tensors (the device check is
tested by itself), and a call past its checks can only report MOE_ERR_CUDA."""
import ctypes

import pytest
import torch

from combine_moe_plan_gb300 import build as moe_build
from combine_moe_plan_gb300 import moe

T, H, E, P, K = 8, 256, 16, 18, 4


@pytest.fixture
def pool(monkeypatch):
    """A Pool over an address that nothing reads."""
    moe_build.build()
    p = moe.Pool.__new__(moe.Pool)
    p.desc = moe.Desc(64, H, E, P, K, 128, 2)
    p.T_max, p.H, p.E, p.P, p.k, p.n_sets = 64, H, E, P, K, 2
    n, h = ctypes.c_size_t(), ctypes.c_void_p()
    assert moe.lib().moe_pool_bytes(ctypes.byref(p.desc), ctypes.byref(n)) == 0
    assert moe.lib().moe_pool_init(ctypes.byref(p.desc), ctypes.c_void_p(1 << 40), n, ctypes.byref(h)) == 0
    p.handle, p._views = h, {}
    monkeypatch.setattr(moe, "_stream", lambda stream: None)
    return p


@pytest.fixture
def anywhere(monkeypatch):
    monkeypatch.setattr(moe, "_on_gpu", lambda t: True)


def strided(*shape, dtype=torch.float32):
    """A view of this shape and type that skips every second element of a row."""
    return torch.zeros(*shape[:-1], 2 * shape[-1], dtype=dtype)[..., ::2]


def routed(pool, logits=None, bias=None, rep_off=None, rep_ids=None):
    return pool.plan_routed(torch.zeros(T, E) if logits is None else logits, moe.Router(),
                            torch.zeros(E) if bias is None else bias,
                            torch.zeros(E + 1, dtype=torch.int32) if rep_off is None else rep_off,
                            torch.zeros(P, dtype=torch.int32) if rep_ids is None else rep_ids)


def test_plan_routed_takes_what_it_reads(pool, anywhere):
    with pytest.raises(moe.MoeError) as e:
        routed(pool)
    assert e.value.rc == -6  # past every check
    with pytest.raises(moe.MoeError) as e:
        pool.plan_routed(torch.zeros(65, E), moe.Router())
    assert e.value.rc == -2  # more tokens than the pool has


@pytest.mark.parametrize("bad", [
    dict(logits=torch.zeros(T, E, dtype=torch.bfloat16)), dict(logits=torch.zeros(T, E, dtype=torch.float64)),
    dict(logits=torch.zeros(T, E - 1)), dict(logits=torch.zeros(T, E + 1)), dict(logits=torch.zeros(T * E)),
    dict(logits=torch.zeros(E, T).t()), dict(logits=strided(T, E)), dict(bias=torch.zeros(E - 1)),
    dict(bias=torch.zeros(E, dtype=torch.bfloat16)), dict(bias=strided(E)), dict(bias=torch.zeros(1, E)),
    dict(rep_off=torch.zeros(E, dtype=torch.int32)), dict(rep_off=torch.zeros(E + 1, dtype=torch.int64)),
    dict(rep_ids=torch.zeros(P - 1, dtype=torch.int32)), dict(rep_ids=torch.zeros(P, dtype=torch.int64)),
    dict(rep_ids=strided(P, dtype=torch.int32))], ids=lambda b: next(iter(b)))
def test_plan_routed_refuses(pool, anywhere, bad):
    with pytest.raises(ValueError, match=next(iter(bad))):
        routed(pool, **bad)


def test_plan_routed_refuses_host_tensors(pool):
    with pytest.raises(ValueError, match="on the GPU"):
        routed(pool)


def test_dispatch_f8_takes_what_it_reads(pool, anywhere):
    with pytest.raises(moe.MoeError) as e:
        pool.dispatch_f8(torch.zeros(T, H, dtype=torch.bfloat16))
    assert e.value.rc == -9  # past every check of the tensor: nothing is planned
    with pytest.raises(moe.MoeError) as e:
        pool.dispatch_f8(torch.zeros(65, H, dtype=torch.bfloat16))
    assert e.value.rc == -2


@pytest.mark.parametrize("bad", [
    torch.zeros(T, H), torch.zeros(T, H, dtype=torch.float16), torch.zeros(T, H - 128, dtype=torch.bfloat16),
    torch.zeros(T, H + 128, dtype=torch.bfloat16), torch.zeros(T * H, dtype=torch.bfloat16),
    torch.zeros(H, T, dtype=torch.bfloat16).t(), strided(T, H, dtype=torch.bfloat16)], ids=range(7))
def test_dispatch_f8_refuses(pool, anywhere, bad):
    with pytest.raises(ValueError, match="x: want"):
        pool.dispatch_f8(bad)


def test_dispatch_f8_refuses_host_tensors(pool):
    with pytest.raises(ValueError, match="on the GPU"):
        pool.dispatch_f8(torch.zeros(T, H, dtype=torch.bfloat16))


F8, INNER, ROWS = torch.float8_e4m3fn, 128, 6


@pytest.fixture
def experts(monkeypatch):
    """Experts over addresses that nothing reads."""
    moe_build.build()
    e = moe.Experts.__new__(moe.Experts)
    e.P, e.H, e.I = P, H, INNER
    e.weights = moe.ExpertWeights(P, H, INNER, *[ctypes.c_void_p(1 << 41)] * 5)
    e._ref = ctypes.byref(e.weights)
    monkeypatch.setattr(moe, "_stream", lambda stream: None)
    return e


def products():
    """Tensors of both products, by the name of their argument."""
    offsets = torch.zeros(P + 1, dtype=torch.int32)
    h, h_scales = torch.zeros(ROWS, INNER, dtype=F8), torch.zeros(ROWS, 4)
    return {"up": dict(codes=torch.zeros(ROWS, H, dtype=F8), scales=torch.zeros(ROWS, 4), offsets=offsets, h=h,
                       h_scales=h_scales),
            "down": dict(h=h, h_scales=h_scales, offsets=offsets, out=torch.zeros(ROWS, H, dtype=torch.bfloat16))}


HOST = [(call, name) for call, args in products().items() for name in args]


@pytest.mark.parametrize("call,name", HOST)
def test_experts_refuse_a_host_tensor(experts, monkeypatch, call, name):
    args = products()[call]
    monkeypatch.setattr(moe, "_on_gpu", lambda t: t is not args[name])
    with pytest.raises(ValueError, match="on the GPU"):
        getattr(experts, call)(**args)


@pytest.mark.parametrize("call", ["up", "down"])
def test_experts_take_device_tensors(experts, anywhere, call):
    with pytest.raises(moe.MoeError) as e:
        getattr(experts, call)(**products()[call])
    assert e.value.rc == -6  # past every check


@pytest.mark.parametrize("name", ["w13", "s13", "w2", "s2"])
def test_experts_weights_on_the_host(monkeypatch, name):
    w = dict(w13=torch.zeros(P, 2 * INNER, H, dtype=F8), s13=torch.zeros(P, 2 * INNER // 128, H // 128),
             w2=torch.zeros(P, H, INNER, dtype=F8), s2=torch.zeros(P, H // 128, INNER // 128))
    monkeypatch.setattr(moe, "_on_gpu", lambda t: t is not w[name])
    with pytest.raises(ValueError, match="on the GPU"):
        moe.Experts(**w)


class Recorder:
    """A pool that notes its calls."""
    H = H

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a, **k: self.calls.append(name)


@pytest.fixture
def net():
    from combine_moe_plan_gb300 import layer
    n = layer.ExpertLayer.__new__(layer.ExpertLayer)
    n.pool, n.experts, n.router, n.bias, n.rep_off, n.rep_ids = Recorder(), None, moe.Router(), None, None, None
    n.inner = [(None, None)]
    return n


BF = torch.bfloat16


def test_expert_layer_calls_in_order(net, anywhere):
    net(torch.zeros(T, H, dtype=BF), torch.zeros(T, E), torch.zeros(T, H, dtype=BF))
    assert net.pool.calls == ["plan_routed", "dispatch_f8", "experts", "combine"]


@pytest.mark.parametrize("x,y", [
    (torch.zeros(T, H), None), (torch.zeros(T, H - 128, dtype=BF), None), (strided(T, H, dtype=BF), None),
    (torch.zeros(T, H, dtype=BF), torch.zeros(T, H)), (torch.zeros(T, H, dtype=BF), torch.zeros(T - 1, H, dtype=BF)),
    (torch.zeros(T, H, dtype=BF), torch.zeros(T, H - 128, dtype=BF)),
    (torch.zeros(T, H, dtype=BF), strided(T, H, dtype=BF))], ids=range(7))
def test_expert_layer_refuses_and_enqueues_nothing(net, anywhere, x, y):
    with pytest.raises(ValueError, match="x: want" if y is None else "y: want"):
        net(x, torch.zeros(T, E), y)
    assert net.pool.calls == []


def test_expert_layer_refuses_host_tensors(net):
    with pytest.raises(ValueError, match="on the GPU"):
        net(torch.zeros(T, H, dtype=BF), torch.zeros(T, E))
    assert net.pool.calls == []
