"""The plans of the integer 4-bit projections, asked of the library by a
small host program (tests/host_w4g_plan.cpp).  Without a device a product's K
is never shared by a cluster."""
import os
import subprocess
from typing import NamedTuple

from block_scaled_precision_requant_b200 import build

HERE = os.path.dirname(os.path.abspath(__file__))


class Plan(NamedTuple):
    few: int  # 1: the decode kernel, 0: the tensor-core kernel
    rt: int  # decode kernel: tiles of 16 weight rows per item, 8-row activation tiles, warps along K, slots, CTAs
    nt: int
    ks: int
    slots: int
    gemv_grid: int
    bm: int  # tensor-core kernel: activation rows per tile, CTAs along K, CTAs
    split: int
    gemm_grid: int


def compile_planner(folder) -> str:
    lib = build.build()
    exe = os.path.join(str(folder), "plan")
    cuda = os.path.dirname(os.path.dirname(build.nvcc_path()))
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", build.CSRC, "-I", os.path.join(cuda, "include"),
                    os.path.join(HERE, "host_w4g_plan.cpp"), lib, f"-Wl,-rpath,{os.path.dirname(lib)}", "-o", exe],
                   check=True)
    return exe


def plans(exe, cases, sms=148):
    """A Plan for each (rows, n, k, group, experts, grouped, indexed)."""
    text = "".join(" ".join(str(int(v)) for v in c) + f" {sms}\n" for c in cases)
    out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True, timeout=120).stdout
    got = [Plan(*map(int, line.split())) for line in out.splitlines()]
    assert len(got) == len(cases)
    return got
