"""mx_linear's choice of a kernel: which one takes the sizes that the tests use and
the measured ones, so that a changed rule cannot move the tests away from a kernel
unnoticed."""
import os
import shutil
import subprocess

import pytest

from tests.linear_shapes import KERNELS, SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    compiler = shutil.which("g++")
    if compiler is None:
        pytest.skip("needs g++")
    exe = str(tmp_path_factory.mktemp("plan") / "linear_plan_check")
    subprocess.run([compiler, "-O1", "-std=c++17", "-I", os.path.join(ROOT, "microscaling_precision_gemm_amd", "csrc"),
                    os.path.join(ROOT, "tests", "host", "linear_plan_check.cpp"), "-o", exe], check=True)

    def ask(shapes):
        out = subprocess.run([exe], input="".join("%d %d\n" % s for s in shapes), capture_output=True, text=True,
                             check=True)
        return [KERNELS[int(line)] for line in out.stdout.split()]
    return ask


def test_shapes_reach_their_kernels(plan):
    assert set(SHAPES) == set(KERNELS)
    for kernel, shapes in SHAPES.items():
        assert plan(shapes) == [kernel] * len(shapes), kernel


def test_measured_cases(plan):
    from perf import more_operators as P
    cases = {c["name"]: (c["rows"], c["n"]) for c in P.listed() if c["op"] == "linear"}
    got = dict(zip(cases, plan(list(cases.values()))))
    assert got == {"linear_one_token": "direct", "linear_few_tokens": "split 64x64", "linear_residual": "tile 256",
                   "linear_inner": "tile 256"}


def test_ends_of_the_range(plan):
    most = 2 ** 26 - 1
    assert plan([(1, 1), (1, most), (most, 1), (most, 512), (512, most)]) == [
        "direct", "direct", "tile 128", "tile 256", "tile 256"]
