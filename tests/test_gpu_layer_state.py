"""What a buffer set's calls leave behind: which of them may follow which, and
on which stream."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from combine_moe_plan_gb300 import moe  # noqa: E402
from tests.gpu_util import ensure_built  # noqa: E402

H, E, K = 256, 8, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def inputs(T, seed=0):
    g = gen(seed)
    return (torch.randn(T, H, generator=g, device="cuda").bfloat16(), torch.randn(T, E, generator=g, device="cuda"))


def test_an_empty_int8_batch_after_an_e4m3_one():
    """A set whose codes are E4M3 still takes an empty batch: nothing is read."""
    pool = moe.Pool(16, H, E, E, K, n_sets=1)
    x, logits = inputs(5)
    pool.plan(logits)
    pool.dispatch_f8(x)
    pool.plan(logits[:0])
    pool.identity_experts(0)
    pool.dispatch(x[:0])
    pool.identity_experts(0)
    assert pool.combine(0).shape == (0, H)
    # the rows in the set are E4M3 all the same
    pool.plan(logits)
    with pytest.raises(moe.MoeError) as e:
        pool.identity_experts(5)
    assert e.value.rc == -9
    assert pool.check() == 0


def weights(P, inner, seed=1):
    from combine_moe_plan_gb300 import layer
    return layer.random_experts(P, H, inner, seed=seed)


def test_experts_want_the_set_dispatched_in_e4m3():
    """Pool.experts reads E4M3 rows: refused for a set that holds INT8 rows, none
    at all, or those of another number of tokens."""
    pool = moe.Pool(16, H, E, E, K)
    ex = weights(E, 128)
    x, logits = inputs(6)
    h, hs = ex.inner(12)

    def refused(T=6, buf=0):
        with pytest.raises(moe.MoeError) as e:
            pool.experts(ex, T, h, hs, buf=buf)
        assert e.value.rc == -9

    refused()
    for int8 in (lambda: pool.dispatch(x), lambda: pool.dispatch(x, after_plan=True),
                 lambda: pool.plan_dispatch(logits, x),
                 lambda: pool.step_host(logits.cpu().pin_memory(), x.cpu().pin_memory(),
                                        torch.empty(6, H, dtype=torch.bfloat16).pin_memory())):
        pool.plan(logits)
        int8()
        refused()
        pool.plan(logits)
        pool.dispatch_f8(x)
        refused(T=5)
        refused(buf=1)
        pool.experts(ex, 6, h, hs)
    with pytest.raises(moe.MoeError) as e:
        pool.experts(ex, 6, h, hs, buf=2)
    assert e.value.rc == -4
    pool.plan(logits[:0])
    pool.dispatch_f8(x[:0])
    pool.experts(ex, 0, h, hs)
    assert pool.check() == 0 and ex.check() == 0


def busy(ms=100):
    """Keep the current stream busy for about so long."""
    torch.cuda._sleep(int(ms * 2e6))


def test_buffers_made_on_a_busy_stream():
    """Experts.inner leaves nothing behind on the stream it is called on that
    could run after a product on another one."""
    ex = weights(1, 256)
    n = 40
    rows = (torch.randn(n, H, generator=gen(2), device="cuda") * 40).to(torch.float8_e4m3fn)
    scales = torch.full((n, 4), 0.02, device="cuda")
    offsets = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    want = [t.clone() for t in ex.up(rows, scales, offsets, *ex.inner(n))]
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    busy()
    h, hs = ex.inner(n)
    ex.up(rows, scales, offsets, h, hs, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(hs[:, :2], want[1][:, :2]) and bool((hs[:, :2] > 0).any())
    assert torch.equal(h.view(torch.uint8), want[0].view(torch.uint8))
    assert ex.check() == 0


def test_a_layer_made_on_a_busy_stream():
    """An error bit that a call on another stream sets is not wiped by the
    layer's construction."""
    from combine_moe_plan_gb300 import layer
    ex = weights(E, 128)
    x, logits = inputs(6)
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    ids = torch.arange(E, dtype=torch.int32, device="cuda")
    ids[:] = E  # no such expert: every copy is skipped and reported
    y = torch.zeros_like(x)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    # the kernels are loaded by a first layer, and its memory is the next one's: nothing below waits for the GPU
    layer.ExpertLayer(ex, 16, E, K, moe.Router(), rep_off=off, rep_ids=ids)(x, logits, y, stream=other)
    torch.cuda.synchronize()
    busy()
    net = layer.ExpertLayer(ex, 16, E, K, moe.Router(), rep_off=off, rep_ids=ids)
    net(x, logits, y, stream=other)
    torch.cuda.synchronize()
    assert net.check() & moe.DEVERR_REPLICA
