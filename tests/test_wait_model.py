"""The experts' kernels' bounded wait (csrc/wait.h), compiled for the host over
phases whose polls and clock are counted."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_moe_plan_gb300", "csrc")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    assert cxx, "no C++ compiler"
    out = str(tmp_path_factory.mktemp("wait") / "libwait_model.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{CSRC}",
                    os.path.join(ROOT, "tests", "wait_model.cpp"), "-o", out], check=True)
    L = ctypes.CDLL(out)
    for f in (L.wait_limit_ns, L.wait_poll_ns, L.wait_polls):
        f.restype = ctypes.c_longlong
    return L


def run(model, ends=-1, other=-1, later=0):
    out = (ctypes.c_longlong * 7)()
    model.wait_run(ctypes.c_longlong(ends), ctypes.c_longlong(other), later, out)
    return dict(zip(("ok", "ns", "polls", "reads", "later_ns", "later_polls", "later_ok"), out))


def test_a_phase_that_never_ends(model):
    """Within the stated bound: the polls before the clock, the limit, a poll
    that was under way when it ran out."""
    r = run(model)
    poll = model.wait_poll_ns() + 45 + 300  # the longest a poll and a reading of the clock take
    assert r["ok"] == 0
    assert model.wait_limit_ns() <= r["ns"] <= model.wait_limit_ns() + (model.wait_polls() + 3) * poll
    assert model.wait_polls() * model.wait_poll_ns() < model.wait_limit_ns() / 10  # the clock starts early


@pytest.mark.parametrize("later", [1, 56, 100_000])
def test_later_waits_take_a_poll_each(model, later):
    """After one wait has given up, each of the following takes one poll, however
    many there are (a summing warp runs through what is left of its tile)."""
    r = run(model, later=later)
    assert r["later_ok"] == 0 and r["later_polls"] == later
    assert r["later_ns"] <= later * (30 + 45 + model.wait_poll_ns())
    assert model.wait_poll_ns() <= 50_000


def test_another_warp_gives_up(model):
    """A wait under way returns at its next poll once the flag is set."""
    at = 10 * model.wait_poll_ns()
    r = run(model, other=at)
    assert r["ok"] == 0 and r["ns"] <= at + 2 * (model.wait_poll_ns() + 45)


def test_a_phase_that_ends(model):
    """Over already: one look.  Later: when it ends, and without the clock as
    long as that is before the first polls have slept their time."""
    assert run(model, ends=0) == dict(ok=1, ns=30, polls=0, reads=0, later_ns=0, later_polls=0, later_ok=0)
    for ends in (100, 10_000, model.wait_poll_ns() * (model.wait_polls() // 2)):
        r = run(model, ends=ends)
        assert r["ok"] == 1 and r["reads"] == 0 and r["ns"] <= ends + 45
    r = run(model, ends=model.wait_limit_ns() // 2)
    assert r["ok"] == 1 and r["ns"] <= model.wait_limit_ns() // 2 + 400


@pytest.mark.parametrize("written", [0, 1, 5, 15, 16, 17, 40, 64])
def test_only_written_ring_entries_count(model, written):
    """A reader of a ring whose writer has stopped takes the entries it wrote and
    no other, also a round later, when the parity of a barrier that was left
    behind says "over" again."""
    n = 100
    ok = (ctypes.c_ubyte * n)()
    model.ring_run(16, written, n, ok)
    assert list(ok) == [1] * written + [0] * (n - written)
