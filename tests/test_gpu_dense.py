"""The bf16 experts' grouped products and their gradients (moe_dense_*) against a
plain implementation in 64 bits, within derived bounds.

Sums in fp32: a product of two bf16 values is exact, and a sum of K of them takes
at most K roundings or truncations of 2^-23 of the terms' sizes, so it is off by at
most K 2^-23 sum |a b|.  A result in bf16 adds half a step, 2^-8 of the value.
"""
import zlib

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from combine_moe_plan_gb300 import moe  # noqa: E402
from tests.gpu_util import ensure_built  # noqa: E402

F8, BF = torch.float8_e4m3fn, torch.bfloat16
STEP = 2.0 ** -8   # bf16, half a step
TINY = 2.0 ** -133  # half the smallest bf16 value


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def gen(*key):
    g = torch.Generator("cuda")
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def normal(g, *shape, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(BF)


def offsets_of(sizes, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(sizes)]), dtype=torch.int32, device="cuda")


def windows(sizes, first):
    lo = first
    for p, m in enumerate(sizes):
        if m:
            yield p, slice(lo, lo + m)
        lo += m


def poisoned(g, sizes, first, tail, *widths, scale=1.0):
    """Rows of a normal distribution; those of no window are NaN and infinities."""
    n = first + int(sum(sizes)) + tail
    out = []
    for width in widths:
        t = normal(g, n, width, scale=scale)
        t[:first] = float("nan")
        t[n - tail:] = float("inf")
        out.append(t)
    return n, out


def untouched(t, sizes, first, value=7.0):
    last = first + int(sum(sizes))
    return bool((t[:first].float() == value).all() and (t[last:].float() == value).all())


def filled(n, width, dtype):
    return torch.full((n, width), 7.0, device="cuda").to(dtype)


def within(got, want, bound):
    far = ((got.double() - want).abs() - bound).max().item()
    assert far <= 0, far


def check_product(sizes, H, I, which, first=0, tail=0):
    """down and up_backward."""
    P = len(sizes)
    g = gen(tuple(sizes), H, I, which)
    K = I if which == "down" else 2 * I
    n, (a,) = poisoned(g, sizes, first, tail, K)
    w = normal(g, P, H, I, scale=I ** -0.5) if which == "down" else normal(g, P, 2 * I, H, scale=H ** -0.5)
    off = offsets_of(sizes, first)
    out = filled(n, H, BF)
    ex = moe.DenseExperts(w2=w) if which == "down" else moe.DenseExperts(w13=w)
    getattr(ex, "down" if which == "down" else "up_backward")(a, off, out)
    assert ex.check() == 0
    for p, at in windows(sizes, first):
        x, v = a[at].double(), w[p].double() if which == "up" else w[p].double().T
        y, big = x @ v, x.abs() @ v.abs()
        within(out[at], y, K * 2.0 ** -23 * big * (1 + STEP) + y.abs() * STEP + TINY)
    assert untouched(out, sizes, first)
    return ex, a, off, out


def check_up(sizes, H, I, first=0, tail=0, keep=True, extra=0):
    P, G = len(sizes), 2 * I // 128
    g = gen(tuple(sizes), H, I, "u")
    n, (x,) = poisoned(g, sizes, first, tail, H)
    w = normal(g, P, 2 * I, H, scale=2 * H ** -0.5)
    off = offsets_of(sizes, first)
    h = filled(n, I, BF)
    ex = moe.DenseExperts(w13=w)
    codes, scales = filled(n, 2 * I, F8), filled(n, (G + 3) // 4 * 4 + extra, torch.float32)
    ex.up(x, off, h, *((codes, scales) if keep else ()))
    assert ex.check() == 0
    for p, at in windows(sizes, first):
        m = at.stop - at.start
        y = x[at].double() @ w[p].double().T
        ey = H * 2.0 ** -23 * (x[at].double().abs() @ w[p].double().abs().T)
        gate, up, eg, eu = y[:, :I], y[:, I:], ey[:, :I], ey[:, I:]
        silu = gate * torch.special.expit(gate)
        v = silu * up
        # |silu'| < 1.1; exp, add, divide and two products, each off by a few 2^-23
        ev = 1.1 * eg * (up.abs() + eu) + silu.abs() * eu + v.abs() * 8 * 2.0 ** -23 + 1e-37
        within(h[at], v, ev * (1 + STEP) + v.abs() * STEP + TINY)
        if not keep:
            continue
        yg, eyg = y.view(m, G, 128), ey.view(m, G, 128)
        amax, ea = yg.abs().amax(-1), eyg.amax(-1)
        s = scales[at, :G].double()
        within(s, amax / 448, ea / 448 + s * 2.0 ** -22 + 1e-44)
        got = codes[at].double().view(m, G, 128)
        # half an E4M3 step of the code: 2^-4 of its size, 2^-10 below the normal ones; at the value's
        # own error the neighbouring code may be the nearest
        step = torch.maximum(got.abs() * 2.0 ** -4, torch.full_like(got, 2.0 ** -10))
        within(got * s[..., None], yg, s[..., None] * step * (1 + 2.0 ** -3) + eyg +
               yg.abs() * ((ea / amax.clamp_min(1e-300))[..., None] * 2 + 2.0 ** -20))
    assert untouched(h, sizes, first)
    if keep:
        assert untouched(codes, sizes, first) and untouched(scales, sizes, first)
    else:
        assert (codes.float() == 7).all() and (scales == 7).all()
    return ex, x, off, h, codes, scales


def kept_values(g, n, I):
    """Codes and scales as `up` leaves them, of values of a few units."""
    G = 2 * I // 128
    v = 2 * torch.randn(n, G, 128, generator=g, device="cuda")
    v[::5, 0] = 0.0
    amax = v.abs().amax(-1, keepdim=True)
    codes = (v * (448 / amax.clamp_min(1e-30))).reshape(n, 2 * I).to(F8)
    scales = torch.full((n, (G + 3) // 4 * 4), float("nan"), device="cuda")  # padding is never read
    scales[:, :G] = amax[..., 0] / 448
    return codes, scales


def check_down_backward(sizes, H, I, first=0, tail=0):
    P, G = len(sizes), I // 128
    g = gen(tuple(sizes), H, I, "b")
    n, (dout,) = poisoned(g, sizes, first, tail, H, scale=0.1)
    w = normal(g, P, H, I, scale=H ** -0.5)
    codes, scales = kept_values(g, n, I)
    row_gates = torch.rand(n, generator=g, device="cuda")
    off = offsets_of(sizes, first)
    dgu, hg, parts = filled(n, 2 * I, BF), filled(n, I, BF), filled(n, G, torch.float32)
    ex = moe.DenseExperts(w2=w)
    ex.down_backward(dout, codes, scales, row_gates, off, dgu, hg, parts)
    assert ex.check() == 0
    for p, at in windows(sizes, first):
        m = at.stop - at.start
        d = dout[at].double() @ w[p].double()
        ed = H * 2.0 ** -23 * (dout[at].double().abs() @ w[p].double().abs())
        v = codes[at].double() * scales[at, :2 * G].double().repeat_interleave(128, 1)
        gv, u, gate = v[:, :I], v[:, I:], row_gates[at].double()[:, None]
        s = torch.special.expit(gv)
        h = gv * s * u
        # codes times scale, exp, add, divide and up to four products: a dozen roundings of 2^-23 at most; the
        # slope's two terms s and g s (1 - s) are rounded by their own sizes (1 - s cancels: 2^-23 of 1)
        r = 12 * 2.0 ** -23
        slope, rough = s + gv * s * (1 - s), s + gv.abs() * s
        within(hg[at], gate * h, (gate * h).abs() * (STEP + r) + TINY)
        du = gate * d * gv * s
        within(dgu[at, I:], du, (gate * ed * (gv * s).abs() + du.abs() * r) * (1 + STEP) + du.abs() * STEP + TINY)
        dg = gate * d * u * slope
        edg = gate * (ed * (u * slope).abs() + (d.abs() + ed) * u.abs() * rough * r)
        within(dgu[at, :I], dg, edg * (1 + STEP) + dg.abs() * STEP + TINY)
        dh, big = (d * h).view(m, G, 128), ((d.abs() + ed) * h.abs()).view(m, G, 128)
        within(parts[at], dh.sum(-1), (ed * h.abs()).view(m, G, 128).sum(-1) + big.sum(-1) * (r + 128 * 2.0 ** -24) + TINY)
    assert untouched(dgu, sizes, first) and untouched(hg, sizes, first) and untouched(parts, sizes, first)
    return ex, dout, codes, scales, row_gates, off, dgu, hg, parts


def check_grad(sizes, H, I, which, kind, first=0, tail=0):
    P = len(sizes)
    g = gen(tuple(sizes), H, I, which, kind)
    M, N = (2 * I, H) if which == "up" else (H, I)
    n, (a, b) = poisoned(g, sizes, first, tail, M, N)
    off = offsets_of(sizes, first)
    dtype = BF if kind == "bf16" else torch.float32
    before = torch.randn(P, M, N, generator=g, device="cuda").to(dtype)
    dw = before.clone()
    ex = moe.DenseExperts(sizes=(P, H, I))
    getattr(ex, which + "_grad")(a, b, off, dw, accumulate=kind == "add")
    assert ex.check() == 0
    seen = set()
    for p, at in windows(sizes, first):
        seen.add(p)
        m = at.stop - at.start
        x, y = a[at].double(), b[at].double()
        want, bound = x.T @ y, m * 2.0 ** -23 * (x.abs().T @ y.abs())
        if kind == "add":
            want = want + before[p].double()
            bound = bound + want.abs() * 2.0 ** -23
        if kind == "bf16":
            bound = bound * (1 + STEP) + want.abs() * STEP + TINY
        within(dw[p], want, bound + 1e-44)
    for p in set(range(P)) - seen:
        assert torch.equal(dw[p], before[p] if kind == "add" else torch.zeros_like(dw[p])), p
    return ex, a, b, off, dw


SIZES = [[1], [0, 1, 0], [127, 0, 1, 128], [129, 3, 64], [300, 5], [31, 32, 33, 0, 0, 65], [0, 0, 257],
         [1] * 40, [2, 16, 17, 15, 96, 97, 160], [513, 1, 384]]
SHAPES = [(128, 128), (384, 128), (128, 384), (640, 256), (256, 640)]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_up_windows(sizes):
    check_up(sizes, 256, 384)


@pytest.mark.parametrize("which", ["down", "up"])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_product_windows(sizes, which):
    check_product(sizes, 384, 256, which)


@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_down_backward_windows(sizes):
    check_down_backward(sizes, 256, 384)


@pytest.mark.parametrize("kind", ["f32", "add", "bf16"])
@pytest.mark.parametrize("which", ["up", "down"])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_grad_windows(sizes, which, kind):
    check_grad(sizes, 384, 256, which, kind)


@pytest.mark.parametrize("H,I", SHAPES)
def test_shapes(H, I):
    sizes = [70, 0, 129, 1]
    check_up(sizes, H, I, first=5, tail=9, extra=4)
    check_up(sizes, H, I, first=5, tail=9, keep=False)
    for which in ("down", "up"):
        check_product(sizes, H, I, which, first=5, tail=9)
        check_grad(sizes, H, I, which, "f32", first=5, tail=9)
        check_grad(sizes, H, I, which, "bf16", first=3, tail=130)
    check_down_backward(sizes, H, I, first=5, tail=9)


@pytest.mark.parametrize("tail", [1, 15, 16, 17, 47, 63])
def test_grad_windows_next_to_nan(tail):
    """A window's last rows share a tile with rows of another window, here NaN: they have no part in the sums."""
    sizes, H, I = [64 + tail, 40, tail], 256, 128
    g = gen(tail, "nan")
    n = sum(sizes)
    a, b = normal(g, n, 2 * I), normal(g, n, H)
    a[sizes[0]:sizes[0] + 40] = float("nan")
    b[sizes[0]:sizes[0] + 40] = float("inf")
    dw = torch.empty(3, 2 * I, H, device="cuda")
    ex = moe.DenseExperts(sizes=(3, H, I))
    ex.up_grad(a, b, offsets_of(sizes), dw)
    assert ex.check() == 0
    for p, at in ((0, slice(0, sizes[0])), (2, slice(n - tail, n))):
        x, y = a[at].double(), b[at].double()
        within(dw[p], x.T @ y, (at.stop - at.start) * 2.0 ** -23 * (x.abs().T @ y.abs()) + 1e-44)
    assert dw[1].isnan().all()


def test_wide_and_long():
    """Inner sizes of many steps, and windows of several tiles beside empty ones."""
    check_up([700, 0, 3, 260], 2176, 512)
    check_product([700, 0, 3, 260], 512, 1152, "down")
    check_product([700, 0, 3, 260], 512, 1152, "up")
    check_down_backward([700, 0, 3, 260], 2176, 512)
    check_grad([1500, 0, 3, 260], 512, 768, "up", "f32")
    check_grad([1500, 0, 3, 260], 512, 768, "down", "add")


def test_bad_windows_are_skipped_and_reported():
    H, I, P = 128, 128, 4
    g = gen("bad")
    n = 64
    x, w = normal(g, n, H), normal(g, P, 2 * I, H)
    for off in ([0, 16, 70, 70, 70], [0, 30, 10, 40, 64], [-4, 16, 32, 48, 64], [0, 40, 40, 20, 64]):
        t = torch.tensor(off, dtype=torch.int32, device="cuda")
        good, top = [], 0
        for p in range(P):
            good.append(off[p] >= top and off[p + 1] >= off[p] and off[p + 1] <= n)
            top = max(top, off[p])
        ex = moe.DenseExperts(w13=w)
        h = filled(n, I, BF)
        ex.up(x, t, h, *ex.kept(n))
        assert ex.check() == moe.DEVERR_WINDOW
        for p in range(P):
            if good[p] and off[p + 1] > off[p]:
                at = slice(off[p], off[p + 1])
                y = x[at].double() @ w[p].double().T
                v = y[:, :I] * torch.special.expit(y[:, :I]) * y[:, I:]
                assert ((h[at].double() - v).abs() <= 0.01 * v.abs() + 1e-3 * y.abs().amax()).all()
        dw = filled(P * 2 * I, H, torch.float32).view(P, 2 * I, H)
        a = normal(g, n, 2 * I)
        ex = moe.DenseExperts(sizes=(P, H, I))
        ex.up_grad(a, x, t, dw)
        assert ex.check() == moe.DEVERR_WINDOW
        for p in range(P):
            if good[p]:
                at = slice(off[p], off[p + 1])
                u, v = a[at].double(), x[at].double()
                within(dw[p], u.T @ v, n * 2.0 ** -23 * (u.abs().T @ v.abs()) + 1e-44)
            else:
                assert (dw[p] == 0).all()


def test_no_rows():
    H, I, P = 128, 256, 3
    g = gen("none")
    ex = moe.DenseExperts(normal(g, P, 2 * I, H), normal(g, P, H, I))
    empty, off = torch.empty(0, H, dtype=BF, device="cuda"), torch.zeros(P + 1, dtype=torch.int32, device="cuda")
    ex.up(empty, off, torch.empty(0, I, dtype=BF, device="cuda"), *ex.kept(0))
    ex.down(torch.empty(0, I, dtype=BF, device="cuda"), off, empty)
    for dtype, accumulate in ((torch.float32, False), (BF, False), (torch.float32, True)):
        dw = torch.full((P, 2 * I, H), 3.0, dtype=dtype, device="cuda")
        ex.up_grad(torch.empty(0, 2 * I, dtype=BF, device="cuda"), empty, off, dw, accumulate)
        assert (dw == (3 if accumulate else 0)).all()
        # rows, but every window empty
        dw.fill_(3)
        ex.up_grad(normal(g, 9, 2 * I), normal(g, 9, H), off, dw, accumulate)
        assert (dw == (3 if accumulate else 0)).all()
    assert ex.check() == 0


def test_many_experts():
    """Up to the most experts: windows of 0 to 2 rows."""
    for P in (385, 700, 4096):
        g = gen(P)
        sizes = torch.randint(0, 3, (P,), generator=torch.Generator().manual_seed(P)).tolist()
        H = I = 128
        n = sum(sizes)
        w = normal(g, P, H, I, scale=0.1)
        a, out = normal(g, n, I), torch.empty(n, H, dtype=BF, device="cuda")
        ex = moe.DenseExperts(w2=w)
        ex.down(a, offsets_of(sizes), out)
        dw = torch.empty(P, H, I, device="cuda")
        ex.down_grad(out, a, offsets_of(sizes), dw)
        assert ex.check() == 0
        owner = torch.arange(P, device="cuda").repeat_interleave(torch.tensor(sizes, device="cuda"))
        x, v = a.double(), w.double()[owner]
        y, big = torch.einsum("ri,rhi->rh", x, v), torch.einsum("ri,rhi->rh", x.abs(), v.abs())
        within(out, y, I * 2.0 ** -23 * big * 1.01 + y.abs() * STEP + TINY)
        want = torch.zeros(P, H, I, dtype=torch.float64, device="cuda")
        want.index_add_(0, owner, out.double()[:, :, None] * x[:, None, :])
        within(dw, want, 4 * 2.0 ** -23 * want.abs() + 2.0 ** -22 * 100)


def test_repeated_calls_and_streams_give_the_same_bits():
    sizes, H, I = [200, 0, 33, 129], 256, 384
    ex, x, off, h, codes, scales = check_up(sizes, H, I)
    again = torch.empty_like(h), torch.empty_like(codes), torch.empty_like(scales)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s):
        ex.up(x, off, *again, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(again[0], h) and torch.equal(again[1].view(torch.uint8), codes.view(torch.uint8))
        assert torch.equal(again[2][:, :6], scales[:, :6])
    ex, a, b, off, dw = check_grad(sizes, H, I, "up", "f32")
    other = torch.empty_like(dw)
    ex.up_grad(a, b, off, other)
    assert torch.equal(dw, other)


def test_small_values_and_zero_rows():
    """Groups of zeros, of values near the smallest, and rows of zeros."""
    H, I, n = 128, 128, 8
    g = gen("small")
    x = normal(g, n, H)
    x[0] = 0
    x[1] *= 2.0 ** -60
    x[2] *= 2.0 ** -120
    w = normal(g, 1, 2 * I, H, scale=0.1)
    ex = moe.DenseExperts(w13=w)
    h, (codes, scales) = torch.empty(n, I, dtype=BF, device="cuda"), ex.kept(n)
    ex.up(x, offsets_of([n]), h, codes, scales)
    assert ex.check() == 0
    assert (h[0] == 0).all() and (codes[0].float() == 0).all() and (scales[0, :2] == 0).all()
    y = x.double() @ w[0].double().T
    back = codes.double() * scales[:, :2].double().repeat_interleave(128, 1)
    big = y.view(n, 2, 128).abs().amax(-1).repeat_interleave(128, 1)
    assert ((back - y).abs() <= y.abs() * 2.0 ** -4 * 1.01 + big / 448 * 2.0 ** -9 + 1e-42).all()


def test_far_gates():
    """Gate values whose exponentials overflow or vanish: finite results, the limits."""
    H, I, n = 128, 128, 4
    codes = torch.zeros(n, 2 * I, device="cuda")
    codes[:, :I] = torch.tensor([448.0, -448.0, 1.0, -1.0], device="cuda")[:, None]
    codes[:, I:] = 2.0
    scales = torch.ones(n, 4, device="cuda")
    scales[2:, 0] = 1e30
    w = torch.zeros(1, H, I, dtype=BF, device="cuda")
    w[0].fill_diagonal_(1.0)
    dout = torch.ones(n, H, dtype=BF, device="cuda")
    dgu, hg, parts = filled(n, 2 * I, BF), filled(n, I, BF), filled(n, 1, torch.float32)
    ex = moe.DenseExperts(w2=w)
    ex.down_backward(dout, codes.to(F8), scales, torch.ones(n, device="cuda"), offsets_of([n]), dgu, hg, parts)
    assert ex.check() == 0
    assert dgu.isfinite().all() and hg.isfinite().all() and parts.isfinite().all()
    assert (hg[0] == 896).all() and (hg[1] == 0).all() and (hg[3] == 0).all()
    assert (dgu[0, :I] == 2).all() and (dgu[0, I:] == 448).all() and (dgu[1] == 0).all() and (dgu[3] == 0).all()


@pytest.mark.parametrize("seed", range(24))
def test_random_windows(seed):
    """Sizes, window lengths (skewed, many of them empty), rows in front and behind drawn at random; average
    windows on both sides of 128 rows, where the products change their form."""
    r = np.random.default_rng(seed)
    H, I = (128 * int(r.integers(1, 9)) for _ in range(2))
    P = int(r.choice([1, 2, 3, 7, 20, 64, 400]))
    mean = float(r.choice([0.5, 4, 30, 120, 150, 400]))
    weight = r.gamma(0.7, size=P)
    sizes = r.poisson(mean * P * weight / weight.sum()) if P * mean < 20000 else r.poisson(mean / 20, size=P)
    sizes = [int(n) for n in sizes]
    if sum(sizes) == 0:
        sizes[-1] = 1
    first, tail = int(r.integers(0, 40)), int(r.integers(0, 200))
    if P > 64:
        H = I = 128
    check_up(sizes, H, I, first, tail, keep=bool(seed % 3))
    check_product(sizes, H, I, "down", first, tail)
    check_product(sizes, H, I, "up", first, tail)
    check_down_backward(sizes, H, I, first, tail)
    check_grad(sizes, H, I, "up", "f32", first, tail)
    check_grad(sizes, H, I, "down", ("add", "bf16")[seed % 2], first, tail)


def test_offsets_past_32_bits():
    """Rows and codes of more than 2^31 elements, the windows at the end of them."""
    H, I, n = 2048, 1024, 1_100_000
    g = gen("far")
    sizes, first = [200, 0, 100], n - 300
    off = offsets_of(sizes, first)
    x = torch.empty(n, H, dtype=BF, device="cuda")
    x[first:] = normal(g, 300, H)
    ex = moe.DenseExperts(normal(g, 3, 2 * I, H, scale=H ** -0.5), normal(g, 3, H, I, scale=H ** -0.5))
    h, (codes, scales) = torch.empty(n, I, dtype=BF, device="cuda"), ex.kept(n)
    ex.up(x, off, h, codes, scales)
    near = offsets_of(sizes)

    def same(far, close):
        assert torch.equal(far[first:].view(torch.uint8), close.view(torch.uint8))

    h2, (codes2, scales2) = torch.empty(300, I, dtype=BF, device="cuda"), ex.kept(300)
    ex.up(x[first:], near, h2, codes2, scales2)
    same(h, h2)
    same(codes, codes2)
    same(scales, scales2)
    gates = torch.rand(n, generator=g, device="cuda")
    dgu, hg, parts = (torch.empty(n, w, dtype=t, device="cuda") for w, t in ((2 * I, BF), (I, BF), (I // 128, torch.float32)))
    dgu2, hg2, parts2 = (t[:300].clone() for t in (dgu, hg, parts))
    ex.down_backward(x, codes, scales, gates, off, dgu, hg, parts)
    ex.down_backward(x[first:], codes2, scales2, gates[first:].contiguous(), near, dgu2, hg2, parts2)
    same(dgu, dgu2)
    same(hg, hg2)
    same(parts, parts2)
    dw, dw2 = (torch.empty(3, 2 * I, H, device="cuda") for _ in range(2))
    ex.up_grad(dgu, x, off, dw)
    ex.up_grad(dgu2, x[first:], near, dw2)
    assert torch.equal(dw, dw2)
    out, out2 = torch.empty(n, H, dtype=BF, device="cuda"), torch.empty(300, H, dtype=BF, device="cuda")
    ex.up_backward(dgu, off, out)
    ex.up_backward(dgu2, near, out2)
    same(out, out2)
    ex.down(hg, off, out)
    ex.down(hg2, near, out2)
    same(out, out2)
    assert ex.check() == 0


def test_gradients_past_32_bits():
    """Gradients of more than 2^31 elements: the last experts', and zeros in between."""
    P, H, I = 1100, 1024, 1024
    g = gen("far grads")
    sizes = [3] + [0] * (P - 3) + [70, 5]
    a, b = normal(g, 78, 2 * I), normal(g, 78, H)
    dw = torch.full((P, 2 * I, H), 7.0, device="cuda")
    ex = moe.DenseExperts(sizes=(P, H, I))
    ex.up_grad(a, b, offsets_of(sizes), dw)
    assert ex.check() == 0
    for p, at in windows(sizes, 0):
        x, y = a[at].double(), b[at].double()
        within(dw[p], x.T @ y, (at.stop - at.start) * 2.0 ** -23 * (x.abs().T @ y.abs()) + 1e-44)
    assert not dw[1:P - 2].any()


def test_more_experts_than_every_stage_has_room_for():
    """The prefix of the windows takes a stage's room: every product, in both forms (a long window among short ones)."""
    sizes = torch.randint(0, 3, (700,), generator=torch.Generator().manual_seed(1)).tolist()
    for long in (0, 100_000):
        sizes[350] = long
        H = I = 128
        check_up(sizes, H, I)
        check_product(sizes, H, I, "down")
        check_product(sizes, H, I, "up")
        check_down_backward(sizes, H, I)
        check_grad(sizes, H, I, "up", "f32")
