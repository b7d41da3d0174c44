"""moe_plan_routed against a plain implementation in 64 bits: ids and placement
equal, gates within a derived bound."""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from combine_moe_plan_gb300 import moe  # noqa: E402
from tests.gpu_util import ensure_built  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def reference(logits, bias, k, score, n_group, topk_group, group_top, renorm, scale):
    """ids [T, k] and gates [T, k] in 64 bits.  The scores and choices that
    experts are compared by are binary32 numbers by definition: computed in 64
    bits and rounded."""
    x = logits.astype(np.float64)
    T, E = x.shape
    with np.errstate(invalid="ignore", over="ignore"):
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-x))
        else:
            e = np.exp(x - x.max(1, keepdims=True))
            s = e / e.sum(1, keepdims=True)
    s = np.nan_to_num(s, nan=0.0)
    s32 = s.astype(np.float32)
    c = (s32 if bias is None else s32 + bias).astype(np.float64)
    if n_group > 1:
        g = c.reshape(T, n_group, E // n_group)
        best = -np.sort(-g, axis=2)[:, :, :group_top].sum(2)
        keep = np.argsort(-best, axis=1, kind="stable")[:, :topk_group]
        kept = np.zeros((T, n_group), bool)
        np.put_along_axis(kept, keep, True, 1)
        # experts of the other groups come after every allowed one, a bias of -inf included
        order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -c, ~np.repeat(kept, E // n_group, 1)), axis=1)
        ids = order[:, :k]
    else:
        ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(s, ids, 1)
    if renorm:
        tot = w.sum(1, keepdims=True)
        w = np.divide(w, tot, out=np.zeros_like(w), where=tot > 0)
    return ids, w * scale


def place(ids, rep_off, rep_ids, P):
    T, k = ids.shape
    if rep_off is None:
        phys = ids
    else:
        n = rep_off[ids + 1] - rep_off[ids]
        phys = rep_ids[rep_off[ids] + np.arange(T)[:, None] % n]
    order = np.argsort(phys.ravel(), kind="stable")
    slot = np.empty(T * k, np.int64)
    slot[order] = np.arange(T * k)
    counts = np.bincount(phys.ravel(), minlength=P)
    return {"topk_e": ids, "phys": phys, "slot": slot.reshape(T, k), "counts": counts,
            "offsets": np.concatenate([[0], np.cumsum(counts)]), "src_token": order // k, "src_k": order % k}


def grid_logits(rng, T, E, top=4.0):
    """Logits on a grid of 1/64: many exact ties, and distinct ones far apart."""
    return (np.round(rng.standard_normal((T, E)).clip(-top, top) * 64) / 64).astype(np.float32)


def gate_bound(logits, k):
    """Relative: exp within 2 ulp, its argument's rounding, add, divide, the sum
    of k terms, the quotient and the factor."""
    span = float(logits[np.isfinite(logits)].max() - logits[np.isfinite(logits)].min())
    return 2.0 ** -24 * (2 * (2 + 2 + 2 * span) + int(np.ceil(np.log2(max(k, 2)))) + 8)


def run(logits, bias, k, rep=(None, None), P=None, buf=0, **router):
    T, E = logits.shape
    P = E if P is None else P
    pool = moe.Pool(max(T, 1), 128, E, P, k, n_sets=2)
    dev = [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (logits, bias, *rep)]
    pool.plan_routed(dev[0], moe.Router(**router), dev[1], dev[2], dev[3], buf=buf)
    v = pool.view(buf)
    assert pool.check() == 0
    n = T * k
    cut = {"topk_e": T, "phys": T, "slot": T, "gates": T, "src_token": n, "src_k": n}
    return {a: v[a][:cut[a]].cpu().numpy() if a in cut else v[a].cpu().numpy()
            for a in ("topk_e", "phys", "slot", "gates", "src_token", "src_k", "counts", "offsets")}


def check(logits, bias, k, rep=(None, None), P=None, buf=0, **router):
    got = run(logits, bias, k, rep, P, buf, **router)
    r = dict(score="sigmoid", n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0) | router
    ids, gates = reference(logits, bias, k, **r)
    want = place(ids, *rep, logits.shape[1] if P is None else P)
    for name, a in want.items():
        np.testing.assert_array_equal(got[name], a, err_msg=name)
    np.testing.assert_allclose(got["gates"], gates, rtol=gate_bound(logits, k), atol=1e-37)
    return got


# (E, n_group): groups that fall on whole lanes, and ones that do not (25, 23 and 11 experts)
SHAPES = [(256, 8), (160, 8), (1024, 32), (96, 4), (48, 6), (16, 2), (32, 32), (100, 4), (299, 13), (33, 3)]


@pytest.mark.parametrize("E,n_group", SHAPES)
@pytest.mark.parametrize("T", [1, 65, 600])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_groups(E, n_group, T, score):
    rng = np.random.default_rng([E, n_group, T])
    size = E // n_group
    for topk_group, group_top, with_bias in ((max(1, n_group // 2), min(2, size), True), (n_group, 1, False)):
        k = min(8, topk_group * size)
        bias = (rng.integers(-200, 200, E) / 1000).astype(np.float32) if with_bias else None
        check(grid_logits(rng, T, E), bias, k, score=score, n_group=n_group, topk_group=topk_group,
              group_top=group_top, renorm=with_bias, scale=2.5, buf=1)


@pytest.mark.parametrize("T", [1, 8, 9, 64, 100, 128, 129, 512, 513, 2049])
@pytest.mark.parametrize("E,k", [(8, 2), (64, 6), (128, 16), (256, 8), (600, 32), (1, 1)])
def test_batch_sizes_without_groups(T, E, k):
    """Both sides of every plan form's limit, 8, 16 and 32 lanes a token."""
    rng = np.random.default_rng([T, E])
    logits = grid_logits(rng, T, E)
    check(logits, None, k, score="sigmoid")
    check(logits, (rng.integers(-50, 50, E) / 1000).astype(np.float32), k, score="softmax", renorm=False, scale=0.5)


@pytest.mark.parametrize("T", [4864, 4865])
@pytest.mark.parametrize("E,k", [(16, 3), (17, 4), (64, 6), (65, 8)])
def test_large_batches(T, E, k):
    """Both sides of the limits between 8 lanes and a warp a token."""
    rng = np.random.default_rng([T, E, 1])
    check(grid_logits(rng, T, E), (rng.integers(-50, 50, E) / 1000).astype(np.float32), k, score="softmax", scale=2.0)


@pytest.mark.parametrize("T", [3, 700])
def test_replicas(T):
    rng = np.random.default_rng(T)
    E, P = 64, 72
    n = np.ones(E, np.int64)
    n[rng.choice(E, P - E, replace=False)] = 2
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    ids = rng.permutation(P).astype(np.int32)
    check(grid_logits(rng, T, E), (rng.integers(-90, 90, E) / 1000).astype(np.float32), 6, (off, ids), P, n_group=8,
          topk_group=3, group_top=2, scale=2.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [5, 530])
def test_masked_logits(score, T):
    """-inf, the type's lowest value, and rows that a mask leaves empty."""
    rng = np.random.default_rng(7)
    E, k = 64, 6
    logits = grid_logits(rng, T, E)
    logits[0::5] = -np.inf
    logits[1::5, : E - 3] = -np.inf
    logits[2::5, 3:] = np.finfo(np.float32).min
    logits[3::5, ::2] = -np.inf
    got = check_masked(logits, None, k, score, 8, 4)
    assert (got["gates"][0::5] == 0).all()
    check_masked(logits, None, k, score, 1, 1)


def check_masked(logits, bias, k, score, n_group, topk_group):
    got = run(logits, bias, k, score=score, n_group=n_group, topk_group=topk_group)
    ids, gates = reference(logits, bias, k, score, n_group, topk_group, 1, True, 1.0)
    np.testing.assert_array_equal(got["topk_e"], ids)
    span = 8.0  # the finite, unmasked logits
    np.testing.assert_allclose(got["gates"], gates, rtol=2.0 ** -24 * (2 * (4 + 2 * span) + 11), atol=1e-37)
    return got


def test_bias_of_minus_infinity_excludes():
    rng = np.random.default_rng(3)
    E, k = 64, 4
    bias = np.zeros(E, np.float32)
    bias[rng.choice(E, 20, replace=False)] = -np.inf
    got = check(grid_logits(rng, 300, E), bias, k, n_group=8, topk_group=4, group_top=1)
    assert np.isfinite(bias[got["topk_e"]]).all()


def test_nan_rows_leave_the_others_alone():
    rng = np.random.default_rng(4)
    logits = grid_logits(rng, 40, 64)
    bad = logits.copy()
    bad[7] = np.nan
    bad[8, ::3] = np.nan
    for score in ("sigmoid", "softmax"):
        a = run(logits, None, 4, score=score, n_group=8, topk_group=4, group_top=2)
        b = run(bad, None, 4, score=score, n_group=8, topk_group=4, group_top=2)
        rest = np.r_[0:7, 9:40]
        np.testing.assert_array_equal(a["topk_e"][rest], b["topk_e"][rest])
        np.testing.assert_array_equal(a["gates"][rest], b["gates"][rest])
        assert (np.sort(b["topk_e"], 1)[:, 1:] > np.sort(b["topk_e"], 1)[:, :-1]).all()
        assert not (b["topk_e"][8] % 3 == 0).any()
        assert np.isfinite(b["gates"]).all()


def test_softmax_choice_does_not_depend_on_the_batch():
    """A token's ids and gates are the same bits alone, in a cluster and in the
    three launches (other lanes a token, other orders of the softmax's sum)."""
    rng = np.random.default_rng(5)
    logits = rng.standard_normal((1500, 64)).astype(np.float32)
    bias = (rng.integers(-20, 20, 64) / 1000).astype(np.float32)
    whole = run(logits, bias, 6, score="softmax", renorm=False)
    for lo, hi in ((0, 1), (10, 90), (100, 600)):
        part = run(logits[lo:hi], bias, 6, score="softmax", renorm=False)
        np.testing.assert_array_equal(part["topk_e"], whole["topk_e"][lo:hi])
        np.testing.assert_array_equal(part["gates"], whole["gates"][lo:hi])


def test_empty_batch():
    got = run(np.zeros((0, 64), np.float32), None, 4)
    assert (got["counts"] == 0).all() and (got["offsets"] == 0).all()


def test_without_clusters():
    """The ticket plan and the three launches take over where clusters are refused."""
    if os.environ.get("MOE_PLAN_NO_CLUSTER") == "1":
        pytest.skip("already without clusters")
    env = dict(os.environ, MOE_PLAN_NO_CLUSTER="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", __file__, "-k",
                        "(test_batch_sizes and (64-8 or 128-256 or 512-600)) or (test_groups and 65) or test_replicas"],
                       env=env, capture_output=True, text=True, timeout=600,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
