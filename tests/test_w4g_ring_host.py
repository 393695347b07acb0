"""The copy rings of the integer 4-bit projection kernels (csrc/w4g_ring.h),
run on the host with late copies and a reader whose wait runs out
(tests/host_w4g_ring.cpp): no barrier is armed twice in a phase, no slot is
written under a copy, and no copy is in flight when the loader ends.  The
path is not run on a GPU, where a wait runs out only after a fault."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "block_scaled_precision_requant_b200", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    out = tmp_path_factory.mktemp("ring") / "libring.so"
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC,
                    os.path.join(HERE, "host_w4g_ring.cpp"), "-o", str(out)], check=True)
    so = ctypes.CDLL(str(out))

    def run(uses, slots, give_up, seed, drain=1, keep_releasing=False):
        got = (ctypes.c_long * 4)()
        so.run_ring(uses, slots, give_up, seed, drain, int(keep_releasing), got)
        return list(got)

    return run


SHAPES = [(1, 3), (3, 3), (4, 6), (6, 6), (7, 6), (40, 3), (41, 4), (95, 12)]


@pytest.mark.parametrize("drain", [1, 2])
@pytest.mark.parametrize("uses,slots", SHAPES)
def test_every_use_is_read(ring, uses, slots, drain):
    for seed in range(30):
        assert ring(uses, slots, uses, seed, drain) == [0, 0, 0, uses]


@pytest.mark.parametrize("drain", [1, 2])
@pytest.mark.parametrize("uses,slots", SHAPES)
def test_a_reader_that_gives_up_leaves_nothing_in_flight(ring, uses, slots, drain):
    for give_up in range(uses):
        for seed in range(20):
            overruns, onto, flying, read = ring(uses, slots, give_up, seed, drain)
            assert (overruns, onto, flying) == (0, 0, 0) and read == give_up


def test_the_model_sees_both_faults(ring):
    """The same ring with the loader waiting only after a wait of its own ran
    out leaves copies in flight; with a reader that goes on releasing, slots
    are armed under a copy."""
    assert any(ring(4, 6, 0, seed, drain=0)[2] for seed in range(20))
    again = [ring(40, 3, 5, seed, keep_releasing=True) for seed in range(50)]
    assert any(r[0] for r in again) and any(r[1] for r in again)


def test_the_kernels_follow_the_rules():
    """The tensor-core kernel's loader always waits for its copies.  The decode
    kernel's does after every warp has met it, if any gave up; a warp that gave
    up releases nothing."""
    def source(name):
        return re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read()))

    gemm, gemv = source("w4g_gemm.cu"), source("w4g_gemv.cu")
    assert gemm.count("drain_ring(") == gemv.count("drain_ring(") == 1
    assert re.search(r"p\.next\(stages\); } } if \(lane == 0\) drain_ring\(it, ", gemm)
    assert re.search(r"__syncwarp\(\); warps_done\(\); if \(lane < kWarps && \*abort_flag\) { [^{}]*drain_ring\(issued, ", gemv)
    assert gemv.count("warps_done();") == 2
    assert gemv.count("mbar_arrive(&released[") == 1 and "if (lane == 0 && !dead) mbar_arrive(&released[slot]);" in gemv
