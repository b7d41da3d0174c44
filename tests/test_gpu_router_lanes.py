"""moe_plan_routed with every number of lanes a token: the same bits, and right
against the plain implementation in 64 bits; and without clusters.

Lanes: a warp a token in a cluster or ticket plan, in three launches with groups,
more than 64 experts, or 17 to 64 up to 4864 tokens; else 8 (k up to 8) or 16.
"""
import os
import re
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from tests.gpu_util import ensure_built  # noqa: E402
from tests.test_gpu_router import check, grid_logits, run  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


# Rows of 64 logits (binary32, big-endian) whose softmax sum, taken in double the
# precision, falls on different sides of a rounding boundary in the order of 32
# lanes and in that of 8.
ROWS = [
    "4062afa940c2dd783fdf7740c079ac56403aabf9409a847040bad0a83ff90828c09de2e0c0e2c1283e223c7cc0dc6e9940e9cc8c"
    "40d97a1bc06dae57413bf1833d8ed24e40a5555140212c12c1190d1b415d1d5ac0352edbc0ab98de3fed0588c123a77f407f9926"
    "403f905040a16f1440fe0fea40afd9ec413d42a5bf75a204c0f045063ff2997c40e5942a40c3d59fbe4eb82d408148173f93cb04"
    "3f5ea47f40979aba4118720240d0cb9cc11d9387c0a00bc9bf2ff850411ff505400b8302c1015b4440618900bfb29fbec1222f53"
    "c0c81b7a3feee0b13e04ff0dc04beb1bc101871cc04ae0863f74d148bf9c7fae3ea70f564049cb004122f676400da0ae",
    "3f798452be3093b03ea8e3edc14fa2c6413c0ec0405cd1083f5bc9e2c12a5052c05d1f8d407db5c2c092a37cbffbdf6a412e8910"
    "4163136e4107d1c2c0d84d9e408e0f61c01d9f5ac1070b0ebfb647a5c05cc4c7c06e612540524eba402c0a50c0a15db74135d1fa"
    "bef28947c137f73ac10d77bdc0135b8e3f01c5bebff8cbf6c071b21a408d64dc3faf8f83bd1a8c30c00160febd36bf9ec0be1ba5"
    "3dd923c0415a474ebf5100103fa5349a3eda118fbfe19a3c40873b5bc13035b740960857c0fcb11cc0617c60c112b762c09af6b4"
    "40e2a1c9401c2a26bfac5b24bfce7360c02e38fc40c44d3f3fbcf68dc076883040e09814c08f0250413975b840368004",
    "40f832d140992e12bfcf17854127369dc13d97c6c077d7ed40b1c786c01bc7cf40e177c640a1c272415c0d67c1658cd84147b705"
    "40e2a296c02a8624c126649fbf985b5640fd6ac2c136a9e0411081754161c2674047445840e36764c08321a2409907a1c11f25f6"
    "40016878c071f77fc0234c90409b2d8a4021176440911c70c0ef3888bff15a4cbed22bccc0f8048640fea681c12cba7840c95486"
    "c02b9a7a3f9dbe7b3f3d8a13c05a96bbc00669d841335c9ac0d32f0cbf0964cc409bf8164115994fc1172528beca766740be8270"
    "3ede06583ff074c1c10d645540ca3c6641394b58410ccc3fc09defcfc0d4cef03f87686dbf58c86c405d321e3fd5df7a",
    "bf68a0b8c128d74cc0a1c7f4c011839e409e4c6940445cd83ea5484640894cccbfaeb2ea3ece3fc2bfdceae33f37fa6cbed2ce32"
    "40933d15c0ebfc06c07016dd3fa4dffc4099f9cec083aa4a3f65ec4b412ab61c412ea3063fe5cbb7bf48454e3f36000b412daa49"
    "3fbd3c5e402b30fd4127e55c406313a23fbb699040e3cddbc0c57e1ec009f3f83da7949dc0a17821c161e595418392d241028cb3"
    "406c7e8cc02f9135c097c41240711606c095adaac068c893c0c125bac048326c40b03e973f454afbc05b1edabfee9c23c12c079e"
    "c0a6aada4180c21dbf922af640b58c15bf99d57d404ec745c0ced8f63e5bb61ec00d70dac14c91ef4037a5ec405f97eb",
]


def hard_rows():
    return np.stack([np.frombuffer(bytes.fromhex(r), ">f4").astype(np.float32) for r in ROWS])


def same_alone(whole, logits, bias, k, spans, **router):
    got = run(whole, bias, k, score="softmax", **router)
    for lo, hi in spans:
        part = run(whole[lo:hi], bias, k, score="softmax", **router)
        np.testing.assert_array_equal(part["topk_e"], got["topk_e"][lo:hi])
        np.testing.assert_array_equal(part["gates"], got["gates"][lo:hi])


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("k", [6, 12])  # 8 and 16 lanes a token in the whole batch, 32 in its parts
def test_softmax_sum_does_not_depend_on_the_lanes(k, renorm):
    rng = np.random.default_rng(k)
    logits = (rng.standard_normal((5000, 64)) * 6).astype(np.float32)
    hard = hard_rows()
    at = [3, 1700, 1701, 4900]
    logits[at] = hard
    bias = (rng.integers(-20, 20, 64) / 1000).astype(np.float32)
    for b in (None, bias):
        same_alone(logits, logits, b, k, [(3, 4), (1700, 1702), (4900, 4901), (0, 100), (4500, 5000), (100, 3000)],
                   renorm=renorm)


@pytest.mark.parametrize("E,k", [(16, 2), (16, 12), (9, 3)])
def test_few_experts_do_not_depend_on_the_lanes(E, k):
    """8 or 16 lanes from 513 tokens on, 32 below."""
    rng = np.random.default_rng([E, k])
    logits = (rng.standard_normal((700, E)) * 6).astype(np.float32)
    same_alone(logits, logits, (rng.integers(-20, 20, E) / 1000).astype(np.float32), k, [(0, 512), (512, 700), (9, 10)])


def clear(logits, bias, score, k):
    """Replace rows in which two choices around the first k + 1 are closer than
    their rounding (but not equal: equal logits and biases are ties by
    definition) by the first row without any."""
    x = logits.astype(np.float64)
    if score == "sigmoid":
        s = 1.0 / (1.0 + np.exp(-x))
    else:
        e = np.exp(x - x.max(1, keepdims=True))
        s = e / e.sum(1, keepdims=True)
    c = -np.sort(-(s if bias is None else s + bias), axis=1)[:, :k + 2]
    gap = c[:, :-1] - c[:, 1:]
    # a score is off by less than 2^-20 of itself (its argument spans 8 units); a sum is rounded to 2^-24
    near = ((gap < 2.0 ** -19 * np.abs(c[:, :-1])) & (gap > 0)).any(1)
    if bias is not None:
        near |= (gap == 0).any(1)
    assert not near.all()
    logits[near] = logits[np.argmin(near)]
    return logits


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,T", [(16, 12, 513), (16, 9, 2100), (9, 9, 600), (64, 12, 4865), (40, 16, 5000),
                                   (64, 5, 4865), (17, 8, 4865), (16, 8, 513)])
def test_eight_and_sixteen_lanes(E, k, T, score):
    rng = np.random.default_rng([E, k, T])
    logits = grid_logits(rng, T, E)
    bias = (rng.integers(-50, 50, E) / 1000).astype(np.float32)
    check(clear(logits.copy(), None, score, k), None, k, score=score, scale=2.0)
    check(clear(logits.copy(), bias, score, k), bias, k, score=score, renorm=False)


@pytest.mark.parametrize("T", [5, 600, 5000])
def test_logits_of_plus_infinity(T):
    """As include/moe.h says: every softmax score of such a token is 0 (its gates
    are 0, its ids the lowest); a sigmoid's score is 1.  The others are untouched."""
    rng = np.random.default_rng(T)
    logits = grid_logits(rng, T, 64)
    bad = logits.copy()
    bad[3, 40] = np.inf
    rest = np.r_[0:3, 4:T]
    for renorm in (False, True):
        a = run(logits, None, 4, score="softmax", renorm=renorm)
        b = run(bad, None, 4, score="softmax", renorm=renorm)
        np.testing.assert_array_equal(b["topk_e"][3], np.arange(4))
        np.testing.assert_array_equal(b["gates"][3], 0)
        np.testing.assert_array_equal(b["topk_e"][rest], a["topk_e"][rest])
        np.testing.assert_array_equal(b["gates"][rest], a["gates"][rest])
    b = run(bad, None, 4, score="sigmoid", renorm=False)
    assert b["topk_e"][3][0] == 40 and b["gates"][3][0] == 1.0


# test_gpu_router's cases without groups, by name, that pass the limits of the
# ticket plan (4 tiles of 32 tokens) and of the three launches' small tiles.
NAMES = [f"test_batch_sizes_without_groups[{E}-{k}-{T}]"
         for E, k in ((8, 2), (64, 6), (128, 16), (256, 8), (600, 32), (1, 1)) for T in (1, 64, 128, 129, 512, 513, 2049)]


def test_every_batch_size_without_clusters():
    if os.environ.get("MOE_PLAN_NO_CLUSTER") == "1":
        pytest.skip("already without clusters")
    path = os.path.join(ROOT, "tests", "test_gpu_router.py")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-m", "gpu", *[f"{path}::{n}" for n in NAMES]],
                       env=dict(os.environ, MOE_PLAN_NO_CLUSTER="1"), capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    assert re.search(rf"\b{len(NAMES)} passed", r.stdout), r.stdout[-500:]
