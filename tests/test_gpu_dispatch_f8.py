"""moe_dispatch_f8 bit for bit against the definition in 64 bits."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from combine_moe_plan_gb300 import moe  # noqa: E402
from tests.gpu_util import ensure_built  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def e4m3_bits(q):
    """Nearest E4M3 bytes of 64-bit values with |q| <= 448, ties to even."""
    a = np.abs(q)
    step = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    v = np.rint(a / step) * step                       # the value, exactly
    e = np.where(v >= 2.0 ** -6, np.floor(np.log2(np.maximum(v, 2.0 ** -6))), -6)
    frac = np.where(v >= 2.0 ** -6, v / np.exp2(e) - 1, v / 2.0 ** -6)
    bits = (np.where(v >= 2.0 ** -6, e + 7, 0) * 8 + frac * 8).astype(np.uint8)
    return bits | np.where(np.signbit(q), 0x80, 0).astype(np.uint8)


def reference(x):
    """bytes [T, H] and fp32 scales [T, H / 128] of fp32-held bf16 values x."""
    T, H = x.shape
    v = x.astype(np.float64).reshape(T, H // 128, 128)
    amax = np.abs(v).max(2, keepdims=True)
    q = v * 448.0 / np.where(amax > 0, amax, 1.0)      # exact product, one rounding in 64 bits
    q32 = q.astype(np.float32).astype(np.float64)      # the correctly rounded fp32 quotient
    return e4m3_bits(q32).reshape(T, H), (amax[..., 0].astype(np.float32) / np.float32(448.0))


def run(x, E=8, k=3, buf=1, n_sets=2):
    T, H = x.shape
    pool = moe.Pool(T, H, E, E, k, n_sets=n_sets)
    xd = torch.from_numpy(x).cuda().bfloat16()
    assert (xd.float().cpu().numpy() == x).all()       # x holds bf16 values
    logits = torch.randn(T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(T))
    pool.plan(logits, buf=buf)
    pool.dispatch_f8(xd, buf=buf)
    assert pool.check() == 0
    v = pool.view(buf)
    slot = v["slot"][:T].long()
    codes = v["codes_f8"].view(torch.uint8)[slot.flatten()].view(T, k, H).cpu().numpy()
    scales = v["scales"][slot.flatten()].view(T, k, -1).cpu().numpy()
    return codes, scales, pool


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().float().numpy()


def check(x, **kw):
    codes, scales, _ = run(x, **kw)
    want, want_s = reference(x)
    G = want_s.shape[1]
    for j in range(codes.shape[1]):
        np.testing.assert_array_equal(codes[:, j], want)
        np.testing.assert_array_equal(scales[:, j, :G], want_s)


@pytest.mark.parametrize("T,H", [(1, 128), (3, 384), (65, 640), (97, 7168), (520, 1152)])
def test_random(T, H):
    rng = np.random.default_rng([T, H])
    x = rng.standard_normal((T, H))
    x[rng.random((T, H)) < 0.002] *= 50
    x[0, :128] = 0
    x[-1, -128:] *= 1e-30
    check(bf16(x))


def test_extremes():
    """Zeros of both signs, the smallest subnormal, the largest finite value,
    and groups on both sides of the fast quotient's range."""
    rows = []
    for top in (2.0 ** -133, 2.0 ** -126, 2.0 ** -101, 2.0 ** -100, 1.0, 2.0 ** 118, 2.0 ** 119, 2.0 ** 120, 3.3895314e38):
        r = np.array([top * f for f in (1, -1, 0.5, 1 / 448, 1 / 512, 1 / 1024, 1 / 2048, 3 / 4096, 0.0, -0.0)] * 13)
        rows.append(r[:128])
    rows.append(np.zeros(128))
    rows.append(-np.zeros(128))
    check(bf16(np.stack(rows)), k=1)


def test_every_significand():
    """Every bf16 significand as the group's maximum against every positive
    bf16 value from it down to where codes are zero."""
    x = []
    for m in range(128):
        top = (1 + m / 128) * 4.0
        vals = ((0x4080 + m) - np.arange(20 * 128)).astype(np.uint32) << 16
        vals = vals.view(np.float32)
        assert vals[0] == top
        for lo in range(0, vals.size, 127):
            part = vals[lo:lo + 127]
            x.append(np.concatenate([[top], part, np.zeros(127 - part.size, np.float32)]))
    check(np.asarray(x, np.float32), k=1)


def test_int8_path_is_not_fooled():
    """identity experts read INT8: refused after dispatch_f8, accepted again
    after dispatch."""
    x = bf16(np.random.default_rng(0).standard_normal((5, 256)))
    _, _, pool = run(x)
    with pytest.raises(moe.MoeError) as e:
        pool.identity_experts(5, buf=1)
    assert e.value.rc == -9
    pool.dispatch(torch.from_numpy(x).cuda().bfloat16(), buf=1)
    pool.identity_experts(5, buf=1)
    assert pool.check() == 0
