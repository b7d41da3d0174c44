"""What one CTA of a pair hands to the other: writes published by an arrival
(csrc/tc.cuh), and in the weights' gradients the last rows of ragged windows, beside
windows of NaN, on every SM and many times over."""
import ctypes
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from combine_moe_plan_gb300 import moe  # noqa: E402
from tests.gpu_util import ensure_built  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_an_arrival_publishes_what_was_written_before(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    out = str(tmp_path / "libpair_payload_probe.so")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17", "-shared", "-Xcompiler",
                    "-fPIC", "-cudart", "static", "-I" + os.path.join(ROOT, "combine_moe_plan_gb300", "csrc"),
                    "-I" + os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "pair_payload_probe.cu"), "-o", out],
                   check=True)
    L = ctypes.CDLL(out)
    L.payload_run.argtypes = [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    rounds = 5000
    got = torch.zeros(3, dtype=torch.int64, device="cuda")
    assert L.payload_run(rounds, got.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert got.tolist() == [1, rounds, 0]


def ragged(extra):
    """Windows of every remainder of 64 (some of several stages), each between windows of NaN rows."""
    sizes, good = [], []
    for n in range(1, 64):
        good.append(len(sizes) + 1)
        sizes += [1 + (n * 37) % 61, n + extra * (n % 3)]
    return sizes + [9], good


@pytest.mark.parametrize("kind", ["f32", "add", "bf16"])
@pytest.mark.parametrize("extra", [0, 64, 128])
def test_gradients_of_ragged_windows_beside_nan(extra, kind):
    """Sums as in test_gpu_dense.py: m products' roundings of 2^-23, and one of the result's type.  Repeated under
    load, the same bits each time."""
    ensure_built()
    sizes, good = ragged(extra)
    H, I, P = 640, 384, len(sizes)
    g = torch.Generator("cuda")
    g.manual_seed(extra)
    n = sum(sizes)
    a = torch.randn(n, 2 * I, generator=g, device="cuda").to(torch.bfloat16)
    b = torch.randn(n, H, generator=g, device="cuda").to(torch.bfloat16)
    lo, rows = 0, {}
    for p, m in enumerate(sizes):
        rows[p] = slice(lo, lo + m)
        if p not in good:
            a[rows[p]], b[rows[p]] = float("nan"), float("inf")
        lo += m
    offsets = torch.tensor([0] + [rows[p].stop for p in range(P)], dtype=torch.int32, device="cuda")
    dtype = torch.bfloat16 if kind == "bf16" else torch.float32
    before = torch.randn(P, 2 * I, H, generator=g, device="cuda").to(dtype)
    ex = moe.DenseExperts(sizes=(P, H, I))
    dw = before.clone()
    ex.up_grad(a, b, offsets, dw, accumulate=kind == "add")
    assert ex.check() == 0
    for p in good:
        x, y, m = a[rows[p]].double(), b[rows[p]].double(), sizes[p]
        want, bound = x.T @ y, m * 2.0 ** -23 * (x.abs().T @ y.abs()) + 1e-44
        if kind == "add":
            want = want + before[p].double()
            bound = bound + want.abs() * 2.0 ** -23
        if kind == "bf16":
            bound = bound * (1 + 2.0 ** -8) + want.abs() * 2.0 ** -8 + 2.0 ** -133
        assert ((dw[p].double() - want).abs() <= bound).all(), (p, m)
    side, load = torch.cuda.Stream(), torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    again = torch.empty_like(dw)
    for _ in range(40):
        with torch.cuda.stream(side):
            load.copy_(load.roll(1))
        again.copy_(before)
        ex.up_grad(a, b, offsets, again, accumulate=kind == "add")
        for p in good:
            assert torch.equal(again[p], dw[p]), p
    torch.cuda.synchronize()
    assert ex.check() == 0
