"""The count of a group's positions, as the adapters' kernels form it, over
offsets of any order and size (compiled for the host; no GPU)."""
import ctypes
import itertools
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "blr_plan.h"
extern "C" int at(int offset, int M) { return blr::plan_at(offset, M); }
extern "C" int rows(int lo, int hi, int M) { return blr::plan_rows(lo, hi, M); }
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    # overflow of a signed integer ends the process
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-ftrapv", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "binary_rank_linear_amd", "csrc"), "-o", str(d / "plan.so"),
                    str(d / "plan.cpp")], check=True)
    return ctypes.CDLL(str(d / "plan.so"))


def test_groups_stay_inside(plan):
    low, high = -2 ** 31, 2 ** 31 - 1
    for M in (1, 2, 64, 600, high - 65536):
        ends = [low, low + 1, -M - 1, -M, -1, 0, 1, M // 2, M - 1, M, min(M + 1, high), high - 1, high]
        for lo, hi in itertools.product(ends, ends):
            a, b = min(max(lo, 0), M), min(max(hi, 0), M)
            assert plan.at(lo, M) == a, (lo, M)
            assert plan.rows(lo, hi, M) == max(b - a, 0), (lo, hi, M)
