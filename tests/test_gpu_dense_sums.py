"""Long sums of the bf16 products against 64 bits: what the tensor cores cut off must
not add up along the inner size.

All values are positive, so that what is cut off has one sign, and rows and columns
have factors of their own, so that the results lie anywhere between two bf16 values.
"""
import zlib

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from combine_moe_plan_gb300 import moe  # noqa: E402
from tests.gpu_util import ensure_built  # noqa: E402

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def positive(*shape, factors):
    """Values of 1 to 2, each row (factors 1) or column (0) times a factor of 1 to 2."""
    g = torch.Generator("cuda")
    g.manual_seed(zlib.crc32(repr((shape, factors)).encode()))
    f = 1 + torch.rand(shape[0] if factors else 1, 1 if factors else shape[1], generator=g, device="cuda")
    return ((1 + torch.rand(*shape, generator=g, device="cuda")) * f).to(BF)


@pytest.mark.parametrize("rows", [128, 700])  # a single CTA's form, and pairs
@pytest.mark.parametrize("which,K", [("down", 65536), ("down", 8192), ("up_backward", 131072), ("up_backward", 8192)])
def test_sums_over_the_longest_inner_sizes(which, K, rows):
    """The mean of the relative errors.  Rounding to bf16 is off by at most 2^-8 either way, uniformly: a root mean
    square of 2^-8 / sqrt 3 at most, of which the mean over n values keeps 1 / sqrt n, four times that at most.  A sum
    of 512 terms in the tensor cores loses at most 2^-23 of itself for each of its 32 steps; adding K / 512 of them up
    to nearest is off by at most 2^-24 each."""
    N = 512
    a = positive(rows, K, factors=1)
    if which == "down":
        w = positive(N, K, factors=1)
        ex, want = moe.DenseExperts(w2=w[None]), a.double() @ w.double().T
    else:
        w = positive(K, N, factors=0)
        ex, want = moe.DenseExperts(w13=w[None]), a.double() @ w.double()
    out = torch.empty(rows, N, dtype=BF, device="cuda")
    getattr(ex, which)(a, torch.tensor([0, rows], dtype=torch.int32, device="cuda"), out)
    assert ex.check() == 0
    off = (out.double() - want) / want
    assert off.abs().max() <= 2.0 ** -8 + K / 16 * 2.0 ** -23
    noise = 4 * 2.0 ** -8 / 3 ** 0.5 / off.numel() ** 0.5
    assert off.mean().abs() <= noise + 32 * 2.0 ** -23 + K / 512 * 2.0 ** -24, off.mean().item()


def normal(key, *shape, scale=1.0):
    g = torch.Generator("cuda")
    g.manual_seed(zlib.crc32(repr((key, shape)).encode()))
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(BF)


def rms(t):
    return t.square().mean().sqrt().item()


@pytest.mark.parametrize("rows,M,N", [(8192, 1024, 256), (1537, 1920, 512), (20000, 256, 256)])
def test_gradients_keep_the_precision_that_the_header_names(rows, M, N):
    """4.5e-7, root mean square over the tensor; at most 6e-6 of the terms' sizes where all have one sign."""
    a, b = normal("a", rows, M), normal("b", rows, N)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    ex = moe.DenseExperts(sizes=(1, M, N))
    dw = torch.empty(1, M, N, device="cuda")
    ex.down_grad(a, b, off, dw)
    want = a.double().T @ b.double()
    assert rms(dw[0].double() - want) <= 4.5e-7 * rms(want)
    ex.down_grad(a.abs(), b.abs(), off, dw)
    want = a.abs().double().T @ b.abs().double()
    assert ((dw[0].double() - want).abs() / want).max() <= 6e-6
    assert ex.check() == 0


@pytest.mark.parametrize("rows,H", [(600, 2048), (300, 7168), (200, 65536)])
def test_gate_parts_keep_the_precision_that_the_header_names(rows, H):
    """8e-7, root mean square over the tensor.  With u = 1 and g = 64 h is 64, and a part 64 times a sum of d."""
    I = 256
    dout, w = normal("d", rows, H), normal("w", 1, H, I, scale=H ** -0.5)
    codes = torch.ones(rows, 2 * I, device="cuda").to(torch.float8_e4m3fn)
    scales = torch.ones(rows, 4, device="cuda")
    scales[:, :2] = 64.0  # silu(64) = 64 to 64 bits
    gates = torch.ones(rows, device="cuda")
    dgu, hg = torch.empty(rows, 2 * I, dtype=BF, device="cuda"), torch.empty(rows, I, dtype=BF, device="cuda")
    parts = torch.empty(rows, I // 128, device="cuda")
    ex = moe.DenseExperts(w2=w)
    ex.down_backward(dout, codes, scales, gates, torch.tensor([0, rows], dtype=torch.int32, device="cuda"), dgu, hg, parts)
    assert ex.check() == 0
    want = 64.0 * (dout.double() @ w[0].double()).view(rows, I // 128, 128).sum(-1)
    assert rms(parts.double() - want) <= 8e-7 * rms(want)
