"""The barriers between the two CTAs of a pair (csrc/tc.cuh) on the GPU: arrivals of
the other CTA end a wait, phase after phase, and a wait that nobody ends is left."""
import ctypes
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIMIT_NS = 20_000_000


def test_arrivals_of_the_other_cta_and_a_wait_that_cannot_end(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    out = str(tmp_path / "libpair_probe.so")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17", "-shared", "-Xcompiler",
                    "-fPIC", "-cudart", "static", f"-DMOE_STALL_NS={LIMIT_NS}ull",
                    "-I" + os.path.join(ROOT, "combine_moe_plan_gb300", "csrc"), "-I" + os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "pair_probe.cu"), "-o", out], check=True)
    L = ctypes.CDLL(out)
    L.pair_run.argtypes = [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    L.pair_polls.restype = ctypes.c_longlong
    rounds = 1000
    got = torch.zeros(8, dtype=torch.int64, device="cuda")
    assert L.pair_run(rounds, got.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    ok, done, left0, left1, time0, time1, poll0, poll1 = got.tolist()
    assert ok == 1 and done == rounds
    assert left0 == 1 and left1 == 1
    # the polls before the clock (twice the longest of eight each), the limit, and the polls around it
    most = (L.pair_polls() + 3) * 2 * max(poll0, poll1) + LIMIT_NS
    print(f"left after {time0 / 1e6:.2f} and {time1 / 1e6:.2f} ms, polls of {poll0 / 1e3:.1f} and {poll1 / 1e3:.1f} us")
    assert LIMIT_NS <= min(time0, time1) and max(time0, time1) <= most
    assert int((torch.ones(4, device="cuda") + 1).sum()) == 8  # the context stays usable
