"""moe_experts_up and moe_experts_down against a plain implementation in 64
bits, within derived bounds.

Sums of fp32: a product of codes is exact; a block of 128 is summed with at
most 128 roundings or truncations of 2^-23 of the terms' sizes, K / 128 blocks
are scaled (two roundings) and added (one each).  So a value y is off by at most
(128 * 2^-23 + (K / 128 + 3) * 2^-24) * sum |a w| in real units.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from combine_moe_plan_gb300 import moe  # noqa: E402
from tests.gpu_util import ensure_built  # noqa: E402

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def gen(*key):
    g = torch.Generator("cuda")
    g.manual_seed(hash(key) % (1 << 31))
    return g


def codes(shape, g):
    """E4M3 codes of a normal distribution with the largest and smallest values among them."""
    c = (60 * torch.randn(shape, generator=g, device="cuda")).clamp(-448, 448)
    c.view(-1)[::97] = 448.0
    c.view(-1)[1::89] = -448.0
    c.view(-1)[2::83] = 2.0 ** -9
    c.view(-1)[3::79] = 0.0
    return c.to(F8)


def rows_of(n, width, g, extra=0):
    stride = (width // 128 + 3) // 4 * 4 + extra
    s = 0.01 * torch.rand(n, stride, generator=g, device="cuda") + 1e-4
    s[:, width // 128:] = float("nan")  # padding is never read
    return codes((n, width), g), s


def weights(P, N, K, g):
    return codes((P, N, K), g), 0.002 * torch.rand(P, N // 128, K // 128, generator=g, device="cuda") + 1e-5


def offsets_of(sizes, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(sizes)]), dtype=torch.int32, device="cuda")


def product(a, sa, w, sw, p):
    """y and sum |a w| of a window, in 64 bits."""
    K = a.shape[1]
    x = a.double() * sa[:, :K // 128].double().repeat_interleave(128, 1)
    v = w[p].double() * sw[p].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    return x @ v.T, x.abs() @ v.abs().T


def slack(K):
    return 128 * 2.0 ** -23 + (K // 128 + 3) * 2.0 ** -24


def check_down(sizes, H, I, first=0, tail=0, extra=0):
    n = first + int(sum(sizes)) + tail
    g = gen(tuple(sizes), H, I)
    a, sa = rows_of(n, I, g, extra)
    w, sw = weights(len(sizes), H, I, g)
    off = offsets_of(sizes, first)
    out = torch.full((n, H), 7.0, dtype=torch.bfloat16, device="cuda")
    ex = moe.Experts(w2=w, s2=sw)
    ex.down(a, sa, off, out)
    assert ex.check() == 0
    lo = first
    for p, m in enumerate(sizes):
        if m:
            y, big = product(a[lo:lo + m], sa[lo:lo + m], w, sw, p)
            bound = big * slack(I) * (1 + 2.0 ** -8) + y.abs() * 2.0 ** -8 + 1e-38
            far = ((out[lo:lo + m].double() - y).abs() / bound).max().item()
            assert far <= 1.0, (p, m, far)
        lo += m
    assert (out[:first] == 7).all() and (out[lo:] == 7).all()  # rows of no window stay
    return a, sa, off, out, ex


def check_up(sizes, H, I, first=0, tail=0, extra=0):
    n = first + int(sum(sizes)) + tail
    g = gen(tuple(sizes), H, I, 1)
    a, sa = rows_of(n, H, g, extra)
    sa = sa * 0.1  # gates of a few units
    w, sw = weights(len(sizes), 2 * I, H, g)
    off = offsets_of(sizes, first)
    G = I // 128
    h = torch.full((n, I), 7.0, device="cuda").to(F8)
    hs = torch.full((n, (G + 3) // 4 * 4 + extra), 7.0, device="cuda")
    ex = moe.Experts(w13=w, s13=sw)
    ex.up(a, sa, off, h, hs)
    assert ex.check() == 0
    lo = first
    for p, m in enumerate(sizes):
        if m:
            y, big = product(a[lo:lo + m], sa[lo:lo + m], w, sw, p)
            e = big * slack(H)
            gate, up, eg, eu = y[:, :I], y[:, I:], e[:, :I], e[:, I:]
            silu = gate * torch.special.expit(gate)
            v = silu * up
            # |silu'| < 1.1; exp, add, divide and two products in fp32, exp's argument exact
            ev = 1.1 * eg * (up.abs() + eu) + silu.abs() * eu + v.abs() * 8 * 2.0 ** -23 + 1e-37
            vg, evg = v.view(m, G, 128), ev.view(m, G, 128)
            amax, ea = vg.abs().amax(-1), evg.amax(-1)
            s = hs[lo:lo + m, :G].double()
            assert ((s - amax / 448).abs() <= ea / 448 + s * 2.0 ** -22 + 1e-44).all(), (p, m)
            got = h[lo:lo + m].double().view(m, G, 128)
            # half an E4M3 step of the code: 2^-4 of its size, 2^-10 below the normal ones; at the
            # value's own rounding error the neighbouring code may be the nearest
            step = torch.maximum(got.abs() * 2.0 ** -4, torch.full_like(got, 2.0 ** -10))
            bound = s[..., None] * step * (1 + 2.0 ** -3) + evg + vg.abs() * (ea / amax.clamp_min(1e-300))[..., None] * 2
            assert ((got * s[..., None] - vg).abs() <= bound + vg.abs() * 2.0 ** -20).all(), (p, m)
        lo += m
    assert (h.float()[:first] == 7).all() and (h.float()[lo:] == 7).all()
    assert (hs[:first] == 7).all() and (hs[lo:] == 7).all()
    return a, sa, off, h, hs, ex


SIZES = [[1], [0, 1, 0], [127, 0, 1, 128], [129, 3, 64], [300, 5], [31, 32, 33, 0, 0, 65], [0, 0, 257],
         [1] * 40, [2, 16, 17, 15, 96, 97, 160], [513, 1, 384]]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_down_windows(sizes):
    check_down(sizes, 384, 256)


@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_up_windows(sizes):
    check_up(sizes, 256, 384)


@pytest.mark.parametrize("H,I", [(128, 128), (256, 128), (128, 640), (1152, 896), (640, 1408), (7168, 256), (384, 2048)])
def test_sizes(H, I):
    check_down([70, 0, 140], H, I)
    check_up([70, 0, 140], H, I)


def test_rows_of_no_window_and_wide_scale_rows():
    check_down([5, 200], 256, 384, first=11, tail=300, extra=4)
    check_up([5, 200], 256, 384, first=11, tail=300, extra=8)


def test_no_rows_at_all():
    check_down([0, 0, 0], 128, 256, tail=9)
    check_up([0, 0, 0], 128, 256, tail=9)
    w, sw = weights(2, 256, 128, gen(0))
    ex = moe.Experts(w2=w, s2=sw)
    a, sa = rows_of(3, 128, gen(1))
    ex.down(a[:0], sa[:0], offsets_of([0, 0]), torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"))
    assert ex.check() == 0


@pytest.mark.parametrize("P", [383, 384, 385, 600, 4096])
def test_many_experts(P):
    """One expert a thread, several, and the most there may be."""
    rng = np.random.default_rng(P)
    sizes = list(rng.integers(0, 4, P))
    check_down(sizes, 128, 128)
    check_up(sizes, 128, 128)


def test_several_threads():
    """Calls of different sizes from four host threads on their own streams."""
    import threading
    jobs = [(check_down, [30, 0, 200], 384, 256), (check_up, [1] * 500, 128, 128), (check_down, [3] * 700, 128, 128),
            (check_up, [129, 64], 256, 640)]
    failed = []

    def work(job):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(3):
                    job[0](*job[1:])
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_bad_windows_are_skipped_and_reported():
    """Windows past the rows, or that run backwards: no access, an error bit,
    the sound windows computed."""
    a, sa, off, out, ex = check_down([40, 50, 60], 256, 128)
    good = out.clone()
    for bad in ([0, 40, 90, 151], [0, 40, 30, 150], [-1, 40, 90, 150], [0, 40, 2**30, 150]):
        out.fill_(7)
        ex.error_word.zero_()
        ex.down(a, sa, torch.tensor(bad, dtype=torch.int32, device="cuda"), out)
        assert ex.check() == moe.DEVERR_WINDOW
        for p in range(3):
            lo, hi = bad[p], bad[p + 1]
            if (lo, hi) == tuple(off[p:p + 2].tolist()):
                assert torch.equal(out[lo:hi], good[lo:hi])
    a, sa, off, h, hs, ex = check_up([40, 50], 256, 128)
    ex.up(a, sa, torch.tensor([0, 40, 91], dtype=torch.int32, device="cuda"), h, hs)
    assert ex.check() == moe.DEVERR_WINDOW


def test_zero_rows_and_columns():
    """Codes that are all zero, scales of zero, a gate far below zero: scale 0 and codes 0."""
    g = gen(9)
    a, sa = rows_of(6, 256, g)
    w, sw = weights(1, 256, 256, g)
    a.view(torch.uint8)[0] = 0
    sa[1, :2] = 0
    w.view(torch.uint8)[0, 128:, :] = 0  # up = 0
    h, hs = moe.Experts(w13=w, s13=sw).up(a, sa, offsets_of([6]), torch.ones(6, 128, device="cuda").to(F8),
                                          torch.ones(6, 4, device="cuda"))
    assert (h.float() == 0).all() and (hs[:, 0] == 0).all()


def test_large_values_do_not_become_nan():
    """Products near the top of fp32 and gates whose exp overflows."""
    g = gen(10)
    a, sa = rows_of(20, 128, g)
    w, sw = weights(1, 256, 128, g)
    h, hs = moe.Experts(w13=w, s13=sw * 1e6).up(a, sa * 1e6, offsets_of([20]), torch.empty(20, 128, device="cuda").to(F8),
                                                torch.zeros(20, 4, device="cuda"))
    assert torch.isfinite(h.float()).all() and torch.isfinite(hs[:, 0]).all()


def test_the_same_bits_again():
    a, sa, off, h, hs, ex = check_up([200, 3, 90], 640, 384)
    h2, hs2 = ex.up(a, sa, off, torch.zeros_like(h), torch.zeros_like(hs))
    assert torch.equal(h.view(torch.uint8), h2.view(torch.uint8)) and torch.equal(hs[:, :3], hs2[:, :3])


def test_another_stream_and_a_graph():
    a, sa, off, out, ex = check_down([33, 140], 384, 256)
    s = torch.cuda.Stream()
    other = torch.zeros_like(out)
    s.wait_stream(torch.cuda.current_stream())
    ex.down(a, sa, off, other, stream=s)
    s.synchronize()
    assert torch.equal(out, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ex.down(a, sa, off, other)
    other.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, other)


@pytest.mark.parametrize("T", [1, 37, 600])
def test_whole_layer(T):
    """plan_routed, dispatch_f8, the experts and combine against the layer in
    64 bits on the dequantised operands."""
    H, I, E, k = 384, 256, 16, 4
    g = gen("layer", T)
    pool = moe.Pool(T, H, E, E, k)
    w13, s13 = weights(E, 2 * I, H, g)
    w2, s2 = weights(E, H, I, g)
    ex = moe.Experts(w13, s13, w2, s2)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    logits = torch.randn(T, E, generator=g, device="cuda")
    pool.plan_routed(logits, moe.Router(n_group=4, topk_group=2, group_top=2, scale=2.5))
    pool.dispatch_f8(x)
    h, hs = ex.inner(T * k)
    pool.experts(ex, T, h, hs)
    y = pool.combine(T)
    assert pool.check() == 0 and ex.check() == 0
    v = pool.view(0)
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    rows = v["codes_f8"].double() * v["scales"][:, :H // 128].double().repeat_interleave(128, 1)
    for e in range(E):
        t, j = (v["topk_e"][:T] == e).nonzero(as_tuple=True)
        r = v["slot"][:T][t, j].long()
        d13 = w13[e].double() * s13[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        d2 = w2[e].double() * s2[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        z = rows[r] @ d13.T
        u = z[:, :I] * torch.special.expit(z[:, :I]) * z[:, I:]
        gate = v["gates"][:T][t, j].double()[:, None]
        want.index_add_(0, t, gate * (u @ d2.T))
        size.index_add_(0, t, gate * (u.abs() @ d2.abs().T))
    # E4M3 between the products: 2^-4 of a value or 2^-10 of a group's scale
    # (at most 2^-10 of its largest value / 448); bf16 after each product.
    assert ((y.double() - want).abs() <= size * (2.0 ** -4 + 2.0 ** -8) + want.abs() * 2.0 ** -7 + size.amax() * 2.0 ** -12).all()


def test_expert_layer_runs_as_calls_and_as_a_graph():
    """ExpertLayer: the same bits call by call, on the other buffer set and from
    a graph; replicas of an expert give what the expert gives."""
    from combine_moe_plan_gb300 import layer
    E, P, H, I, k, T = 8, 10, 256, 256, 2, 70
    ex = layer.random_experts(P, H, I)
    for t in (ex.w13, ex.s13, ex.w2, ex.s2):  # physical 8 and 9 are second copies of 2 and 5
        t.view(torch.uint8)[8] = t.view(torch.uint8)[2]
        t.view(torch.uint8)[9] = t.view(torch.uint8)[5]
    off = torch.tensor([0, 1, 2, 4, 5, 6, 8, 9, 10], dtype=torch.int32, device="cuda")
    ids = torch.tensor([0, 1, 2, 8, 3, 4, 5, 9, 6, 7], dtype=torch.int32, device="cuda")
    router = moe.Router(n_group=2, topk_group=1, group_top=1)
    net = layer.ExpertLayer(ex, T, E, k, router, rep_off=off, rep_ids=ids, n_sets=2)
    g = gen("replicas")
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    logits = torch.randn(T, E, generator=g, device="cuda")
    y = net(x, logits)
    assert net.check() == 0
    assert torch.equal(y, net(x, logits, buf=1))
    single = layer.ExpertLayer(moe.Experts(ex.w13[:8], ex.s13[:8], ex.w2[:8], ex.s2[:8]), T, E, k, router)
    assert torch.equal(y, single(x, logits))
    out = torch.zeros_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        net(x, logits, out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, out)
    with pytest.raises(ValueError):
        net(x[:5], logits)
