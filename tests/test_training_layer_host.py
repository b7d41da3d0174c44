"""layer.TrainingLayer refuses what it cannot take before it enqueues anything.

There is no GPU here: host tensors stand for device tensors, and a pool and experts
that note their calls for the real ones."""
import pytest
import torch

from combine_moe_plan_gb300 import layer, moe

T, H, I, E, P, K = 8, 256, 128, 6, 6, 2
BF = torch.bfloat16


class Recorder:
    """Notes its calls."""

    def __init__(self, calls, **fields):
        self.calls = calls
        self.__dict__.update(fields)

    def __getattr__(self, name):
        if name.startswith("_"):
            raise AttributeError(name)
        return lambda *a, **k: self.calls.append(name)


@pytest.fixture
def net(monkeypatch):
    """A TrainingLayer after a forward of T tokens, whose calls are noted."""
    monkeypatch.setattr(moe, "_on_gpu", lambda t: True)
    monkeypatch.setattr(moe, "_device", lambda: -1)  # where host tensors say they are
    monkeypatch.setattr(layer.TrainingLayer, "_reads", lambda self, stream, *tensors: 0)
    n = layer.TrainingLayer.__new__(layer.TrainingLayer)
    n.calls = []
    n.pool = Recorder(n.calls, T_max=T, H=H, E=E, P=P, k=K, workspace=torch.zeros(1))
    n.experts = Recorder(n.calls, P=P, H=H, I=I, error_word=torch.zeros(1, dtype=torch.int32))
    n.experts._gradient = lambda *a: moe.DenseExperts._gradient(n.experts, *a)
    n.router = n.bias = n.rep_off = n.rep_ids = None
    n.views, n.kept, n.saved, n.logits = [{"offsets": None, "ex_out": None}], [(None, None)], [None], [None]
    n.x_rows = n.d_rows = n.h = n.dgu = n.parts = n.row_gates = None
    n.dgates = torch.zeros(T, K)
    return n


def at(offset, *shape, dtype=torch.float32):
    """A contiguous tensor that begins `offset` elements behind a 16-byte boundary."""
    n = 1
    for s in shape:
        n *= s
    return torch.zeros(n + 64, dtype=dtype)[16 + offset:16 + offset + n].view(*shape)


def kept():
    """What a forward leaves for the backward: x, no logits (there is no router), a stream."""
    return at(0, T, H, dtype=BF), None, 0


def backward_args(**other):
    return {"dy": at(0, T, H, dtype=BF), "dw13": at(0, P, 2 * I, H), "dw2": at(0, P, H, I), "dx": at(0, T, H, dtype=BF),
            "dlogits": at(0, T, E), **other}


def test_backward_calls(net):
    net.saved[0] = kept()
    net.backward(**backward_args())
    assert net.calls == ["scatter", "down_backward", "down_grad", "up_backward", "scatter", "up_grad", "gather",
                         "gates_backward"]
    assert net.saved == [None]


BAD = {"dy": at(1, T, H, dtype=BF), "dx": at(4, T, H, dtype=BF), "dlogits": at(1, T, E), "dw13": at(2, P, 2 * I, H),
       "dw2": at(3, P, H, I)}


@pytest.mark.parametrize("name", BAD)
def test_backward_refuses_odd_addresses_and_enqueues_nothing(net, name):
    """A row slice of a longer buffer: contiguous, but not on a 16-byte boundary."""
    net.saved[0] = saved = kept()
    with pytest.raises(ValueError, match=f"{name}: want"):
        net.backward(**backward_args(**{name: BAD[name]}), accumulate=True)
    assert net.calls == [] and net.saved[0] is saved


@pytest.mark.parametrize("name", BAD)
def test_backward_refuses_tensors_of_another_gpu(net, monkeypatch, name):
    """(Told by the type and shape in the message: host tensors have one place.)"""
    net.saved[0] = kept()
    args = backward_args()
    real = torch.Tensor.get_device
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1 if t is args[name] else real(t))
    with pytest.raises(ValueError, match="current GPU"):
        net.backward(**args, accumulate=True)
    assert net.calls == []


def forward_args(**other):
    return {"x": at(0, T, H, dtype=BF), "logits": at(0, T, E), "y": at(0, T, H, dtype=BF), **other}


def replicas(net, **other):
    net.rep_off = other.get("rep_off", torch.arange(E + 1, dtype=torch.int32))
    net.rep_ids = other.get("rep_ids", torch.arange(P, dtype=torch.int32))


@pytest.mark.parametrize("with_replicas", [False, True])
def test_forward_calls(net, with_replicas):
    if with_replicas:
        replicas(net)
    args = forward_args()
    net.forward(**args)
    assert net.calls == ["plan", "scatter", "up", "down", "combine"]
    assert net.saved[0][0] is args["x"]


@pytest.mark.parametrize("name,bad", [("x", at(1, T, H, dtype=BF)), ("logits", at(2, T, E)), ("y", at(4, T, H, dtype=BF))])
def test_forward_refuses_odd_addresses_and_enqueues_nothing(net, name, bad):
    with pytest.raises(ValueError, match=f"{name}: want"):
        net.forward(**forward_args(**{name: bad}))
    assert net.calls == []


@pytest.mark.parametrize("name", ["x", "logits", "y", "rep_off", "rep_ids", "bias"])
def test_forward_refuses_tensors_of_another_gpu(net, monkeypatch, name):
    replicas(net)
    net.bias = torch.zeros(E)
    args = forward_args()
    there = args.get(name, getattr(net, name, None))
    real = torch.Tensor.get_device
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1 if t is there else real(t))
    with pytest.raises(ValueError, match="current GPU"):
        net.forward(**args)
    assert net.calls == []


@pytest.mark.parametrize("bad", [dict(rep_off=torch.arange(E + 1)), dict(rep_off=torch.zeros(E, dtype=torch.int32)),
                                 dict(rep_ids=torch.arange(P)), dict(rep_ids=torch.zeros(P - 1, dtype=torch.int32)),
                                 dict(rep_ids=torch.zeros(2 * P, dtype=torch.int32)[::2])], ids=str)
def test_forward_refuses_a_replica_map_that_the_plan_would_misread(net, bad):
    replicas(net, **bad)
    with pytest.raises(ValueError, match=f"{next(iter(bad))}: want"):
        net.forward(**forward_args())
    assert net.calls == []


def test_forward_refuses_to_write_over_what_it_keeps(net):
    both = at(0, 2 * T, H, dtype=BF)
    for x, y in ((both[:T], both[:T]), (both[:T], both[T // 2:T // 2 + T]), (both[T // 2:T // 2 + T], both[:T])):
        with pytest.raises(ValueError, match="kept"):
            net.forward(**forward_args(x=x, y=y))
    assert net.calls == []
    net.forward(**forward_args(x=both[:T], y=both[T:]))
    assert net.calls
