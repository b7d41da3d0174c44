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
