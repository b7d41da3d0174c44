"""E4M3 rows split over ranks: dispatch_f8 on every rank, moe_ep_pull into the
owners' receive buffers, the experts' products on those, the rows pulled back and
combined: the bits that a layer holding every expert gives."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from combine_moe_plan_gb300 import ep, layer, moe  # noqa: E402
from tests.gpu_util import ensure_built  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("R,tokens", [(1, [33]), (2, [96, 40]), (3, [1, 200, 17])])
def test_split_products_give_the_layers_bits(R, tokens):
    H, I, E, k = 384, 256, 12, 3
    router = moe.Router("sigmoid", n_group=3, topk_group=2, group_top=2, scale=2.5)
    ex = layer.random_experts(E, H, I, seed=R)
    g = torch.Generator("cuda").manual_seed(R)
    xs = [torch.randn(T, H, generator=g, device="cuda").bfloat16() for T in tokens]
    logits = [torch.randn(T, E, generator=g, device="cuda") for T in tokens]
    net = layer.ExpertLayer(ex, max(tokens), E, k, router)
    want = [net(x, lo) for x, lo in zip(xs, logits)]
    assert net.check() == 0

    group = ep.EmulatedGroup(R, max(tokens), H, E, E, k, cores=8)
    for r in range(R):
        group.pools[r].plan_routed(logits[r], router)
        group.pools[r].dispatch_f8(xs[r])
    counts = group.counts()
    disp, comb, recv_rows = group.schedules(counts)
    group.pull_dispatch(*group.upload(disp))
    parts = []  # kept until the end: the kernels read their weights
    for d in range(R):
        first, n = ep.experts(R, E, d)
        mine = moe.Experts(ex.w13[first:first + n], ex.s13[first:first + n], ex.w2[first:first + n], ex.s2[first:first + n])
        offsets = torch.from_numpy(ep.layout(counts, d)[0]).cuda()
        h, hs = mine.inner(recv_rows[d])
        mine.up(group.recv_codes[d].view(torch.float8_e4m3fn), group.recv_scales[d], offsets, h, hs, rows=recv_rows[d])
        mine.down(h, hs, offsets, group.recv_ex[d], rows=recv_rows[d])
        parts.append((mine, offsets, h, hs))
    group.pull_combine(*group.upload(comb))
    ys = group.combine(tokens)
    torch.cuda.synchronize()
    assert group.check() == 0 and all(p[0].check() == 0 for p in parts)
    for y, w in zip(ys, want):
        assert torch.equal(y, w)
