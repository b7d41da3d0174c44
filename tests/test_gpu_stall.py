"""The experts' kernels' bounded waits (csrc/wait.h, tc.cuh) on the GPU, on an
mbarrier that nobody arrives at."""
import ctypes
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIMIT_NS = 20_000_000


def test_a_wait_that_cannot_end_is_left_and_so_are_the_later_ones(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    out = str(tmp_path / "libstall_probe.so")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17", "-shared", "-Xcompiler",
                    "-fPIC", "-cudart", "static", f"-DMOE_STALL_NS={LIMIT_NS}ull",
                    "-I" + os.path.join(ROOT, "combine_moe_plan_gb300", "csrc"), "-I" + os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "stall_probe.cu"), "-o", out], check=True)
    L = ctypes.CDLL(out)
    L.stall_run.argtypes = [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    L.stall_polls.restype = L.stall_poll_ns.restype = ctypes.c_longlong
    later = 5_000
    got = torch.zeros(9, dtype=torch.int64, device="cuda")
    assert L.stall_run(later, got.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    first, second, later0, later1, ok, any_ok, gave_up, over_ok, over_flag = got.tolist()
    assert (ok, any_ok, gave_up, over_ok, over_flag) == (0, 0, 1, 1, 0)
    # the polls before the clock, the limit, a poll that was under way; the other warp a poll later
    most = (L.stall_polls() + 3) * L.stall_poll_ns() + LIMIT_NS
    print(f"first waits {first / 1e6:.2f} and {second / 1e6:.2f} ms, {2 * later} later ones {later0 / 1e6:.2f} ms")
    assert max(first, second) >= LIMIT_NS and max(first, second) <= most
    # 2 * later waits of one poll each
    assert max(later0, later1) <= 2 * later * (L.stall_poll_ns() + 2000)
    # the context stays usable
    assert int((torch.ones(4, device="cuda") + 1).sum()) == 8
