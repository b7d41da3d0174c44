"""Host-only tests of the scored router's, the E4M3 dispatch's and the experts'
entry points: every refusal comes before a launch (there is no GPU here, so a
call past its checks could only report MOE_ERR_CUDA, -6)."""
import ctypes

import pytest
import torch

from combine_moe_plan_gb300 import build as moe_build
from combine_moe_plan_gb300 import moe

GOOD, ODD = ctypes.c_void_p(1 << 41), ctypes.c_void_p((1 << 41) + 4)


@pytest.fixture(scope="module")
def L():
    moe_build.build()
    return moe.lib()


@pytest.fixture
def pool(L):
    d = moe.Desc(64, 256, 16, 16, 4, 128, 2)
    n = ctypes.c_size_t()
    assert L.moe_pool_bytes(ctypes.byref(d), ctypes.byref(n)) == 0
    h = ctypes.c_void_p()
    assert L.moe_pool_init(ctypes.byref(d), ctypes.c_void_p(1 << 40), n, ctypes.byref(h)) == 0
    yield h
    L.moe_pool_destroy(h)


def _routed(L, pool, router, logits=GOOD, bias=None, T=8, ro=None, ri=None, buf=0):
    return L.moe_plan_routed(pool, None if router is None else ctypes.byref(router), logits, bias, T, ro, ri, buf, None)


@pytest.mark.parametrize("fields", [
    dict(n_group=3), dict(n_group=0), dict(n_group=64), dict(n_group=4, topk_group=0), dict(n_group=4, topk_group=5),
    dict(n_group=8, topk_group=1), dict(n_group=16, topk_group=8, group_top=2), dict(group_top=0), dict(group_top=3),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan"))])
def test_router_out_of_range(L, pool, fields):
    assert _routed(L, pool, moe.Router(**fields)) == -2


def test_router_unknown_score(L, pool):
    r = moe.Router()
    r.score = 2
    assert _routed(L, pool, r) == -2
    with pytest.raises(ValueError):
        moe.Router(score="tanh")


def test_plan_routed_checks_like_plan(L, pool):
    r = moe.Router(n_group=4, topk_group=2, group_top=2)
    assert _routed(L, None, r) == -1
    assert _routed(L, pool, None) == -1
    assert _routed(L, pool, r, T=-1) == -2
    assert _routed(L, pool, r, T=65) == -2
    assert _routed(L, pool, r, buf=2) == -4
    assert _routed(L, pool, r, logits=None) == -1
    assert _routed(L, pool, r, logits=ODD) == -3
    assert _routed(L, pool, r, bias=ODD) == -3
    assert _routed(L, pool, r, ro=GOOD) == -1


def test_dispatch_f8_checks_like_dispatch(L, pool):
    f = L.moe_dispatch_f8
    assert f(pool, GOOD, 8, 0, None) == -9
    assert f(pool, ODD, 8, 0, None) == -3
    assert f(pool, None, 8, 0, None) == -1
    assert f(pool, GOOD, 8, 2, None) == -4
    assert f(pool, GOOD, 65, 0, None) == -2
    assert f(None, GOOD, 8, 0, None) == -1


def _weights(P=4, H=256, I=384, w13=GOOD, s13=GOOD, w2=GOOD, s2=GOOD, err=GOOD):
    return moe.ExpertWeights(P, H, I, w13, s13, w2, s2, err)


def _up(L, w, codes=GOOD, scales=GOOD, stride=4, offsets=GOOD, rows=8, h=GOOD, hs=GOOD, h_stride=4):
    return L.moe_experts_up(None if w is None else ctypes.byref(w), codes, scales, stride, offsets, rows, h, hs,
                            h_stride, None)


def _down(L, w, h=GOOD, hs=GOOD, h_stride=4, offsets=GOOD, rows=8, out=GOOD):
    return L.moe_experts_down(None if w is None else ctypes.byref(w), h, hs, h_stride, offsets, rows, out, None)


@pytest.mark.parametrize("call", [_up, _down])
def test_experts_common_refusals(L, call):
    assert call(L, None) == -1
    assert call(L, _weights(err=None)) == -1
    assert call(L, _weights(err=ODD)) == -3
    for bad in (dict(P=0), dict(P=4097), dict(H=200), dict(H=0), dict(H=65664), dict(I=64), dict(I=130)):
        assert call(L, _weights(**bad)) == -2, bad
    assert call(L, _weights(), rows=-1) == -2
    assert call(L, _weights(), rows=2**31 - 1) == -2
    assert call(L, _weights(), offsets=None) == -1
    assert call(L, _weights(), offsets=ODD) == -3
    assert call(L, _weights(), h_stride=2) == -2    # not whole 16-byte rows
    assert call(L, _weights(I=640), h_stride=4) == -2  # fewer than I / 128
    assert call(L, _weights(), rows=0, h=None, offsets=None) == 0  # no rows: nothing to do


def test_experts_up_refusals(L):
    w = _weights()
    for name in ("codes", "scales", "h", "hs"):
        assert _up(L, w, **{name: None}) == -1, name
        assert _up(L, w, **{name: ODD}) == -3, name
    assert _up(L, w, stride=3) == -2
    assert _up(L, w, stride=0) == -2
    assert _up(L, _weights(w13=None)) == -1
    assert _up(L, _weights(s13=ODD)) == -3


def test_experts_down_refusals(L):
    w = _weights()
    for name in ("h", "hs", "out"):
        assert _down(L, w, **{name: None}) == -1, name
        assert _down(L, w, **{name: ODD}) == -3, name
    assert _down(L, _weights(s2=None)) == -1
    assert _down(L, _weights(w2=ODD)) == -3


def test_binding_checks_tensors():
    """The binding refuses tensors that the call would misread."""
    f8 = torch.float8_e4m3fn
    ok = torch.zeros(4, 8, dtype=f8)
    moe._tensor("x", ok, f8, 4, 8)
    moe._tensor("x", ok, f8, 3)
    for bad in (ok.view(torch.int8), ok.t(), ok[:, :4], ok[:2], ok.view(-1)):
        with pytest.raises(ValueError):
            moe._tensor("x", bad, f8, 4, 8)
    w, s = torch.zeros(2, 256, 128, dtype=f8), torch.zeros(2, 2, 1)
    moe._block_scaled("w2", w, s, 2, 256, 128)
    for bad_w, bad_s in ((w.view(torch.int8), s), (w[:1], s), (w, s[:1]), (w, s.double()), (w.transpose(1, 2), s)):
        with pytest.raises(ValueError):
            moe._block_scaled("w2", bad_w, bad_s, 2, 256, 128)
    with pytest.raises(ValueError):
        moe.Experts()
    with pytest.raises(ValueError):
        moe.Experts(w13=ok)
