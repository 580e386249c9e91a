"""The cases that the GPU tests compare (ff_cases.py) take every kernel that calls of many sizes take, by the
library's own plan: its host header compiled into a small program (ff_plan.cpp).
"""
import os
import subprocess

import pytest

from ff_cases import CASES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("plan") / "ff_plan")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    subprocess.run(["g++", "-O2", "-std=c++17", "-D__HIP_PLATFORM_AMD__=1", f"-isystem{rocm}/include",
                    "-I" + os.path.join(ROOT, "dynamic_dilated_depthwise_amd", "csrc"),
                    os.path.join(ROOT, "tests", "ff_plan.cpp"), "-o", out], check=True)

    def ask(*args, calls=()):
        lines = "\n".join(" ".join(map(str, c)) for c in calls)
        return subprocess.run([out, *args], input=lines, capture_output=True, text=True, check=True, timeout=100).stdout.splitlines()
    return ask


def test_every_kernel_is_compared(plan):
    taken = set()
    for line in plan(calls=CASES):
        taken |= set(line.strip(";").split(";"))
    found = dict(line.split("\t") for line in plan("sweep", "60000", "3e11"))
    assert len(found) > 200
    missing = {k: c for k, c in found.items() if k not in taken}
    assert not missing, "no case of ff_cases.py takes " + "; ".join(f"{k} (as {c} does)" for k, c in missing.items())


def test_large_training_steps(plan):
    """The tiles of a large model's steps are among those that are compared."""
    taken = set(";".join(plan(calls=CASES)).split(";"))
    for call, tiles in ((("bf16", "linear", "none", 16384, 5632, 2048), ("grad_x 256x256", "grad_w 256x256")),
                        (("bf16", "gated", "silu", 16384, 2048, 5632), ("grad_x terms 256x256", "grad_w terms 256x256")),
                        (("f32", "linear", "gelu", 2048, 1024, 2304), ("grad_x 128x128", "grad_w 128x128"))):
        kernels = set(plan(calls=[call])[0].strip(";").split(";"))
        assert all(any(t in k for k in kernels) for t in tiles), kernels
        assert kernels <= taken, kernels - taken
