"""The routing plan on the host: every plan is launchable, and the kernels that
are built are those that a plan can ask for."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_weight_quantization_16_amd", "csrc")


def test_kernels_are_those_that_plans_ask_for(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "route_plan_check")
    subprocess.run([cxx, "-std=c++17", "-O2", "-I", CSRC, os.path.join(ROOT, "tests", "route_plan_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout
    asked = [tuple(map(int, line.split())) for line in out.stdout.splitlines()]
    text = open(os.path.join(CSRC, "moe.hip")).read()
    built = {(int(a), int(b)) for a, b in re.findall(r"GQ_ROUTE\((\d+), (\d+)\)", text)}
    for one in (0, 1):   # one block for all tokens, or many
        assert {(a, b) for a, b, o in asked if o == one} == built
