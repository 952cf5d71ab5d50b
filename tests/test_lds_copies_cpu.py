"""Copies from memory into LDS in the built library's device code.

Such a load takes its LDS address from M0, and gfx9 asks for one wait state
(one instruction in between) after a scalar write of M0.  The sources issue
these loads through inline asm, where the compiler adds no wait states, so the
device code itself is read here.
"""
import os
import re
import shutil
import subprocess

import pytest

from post_weight_quantization_16_amd import build as b

LLVM = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    """One list of instructions for each object of device code in the library."""
    dump = os.path.join(LLVM, "llvm-objdump")
    if not os.path.exists(dump):
        pytest.skip("no llvm-objdump")
    if not os.path.exists(b.LIB):
        b.build()
    tmp = tmp_path_factory.mktemp("device_code")
    lib = shutil.copy(b.LIB, tmp)
    subprocess.run([dump, "--offloading", lib], cwd=tmp, check=True, stdout=subprocess.DEVNULL)
    out = []
    for f in sorted(os.listdir(tmp)):
        if f.endswith(b.ARCH):
            text = subprocess.run([dump, "-d", "--no-show-raw-insn", f], cwd=tmp, check=True,
                                  capture_output=True, text=True).stdout
            out.append([l.split("//")[0].strip() for l in text.splitlines() if l.startswith("\t")])
    assert out
    return out


def test_every_copy_waits_for_its_address(listing):
    copies, early = 0, []
    for code in listing:
        for before, ins in zip(code, code[1:]):
            if re.match(r"(global|buffer)_load_\w*lds|(global|buffer)_load_\w+ .*\blds\b", ins):
                copies += 1
                if re.match(r"s_\w+ m0\b", before):
                    early.append(f"{before}; {ins}")
    assert copies > 100   # the products and the Hessian copy this way
    assert not early, f"{len(early)} of {copies} copies right behind the write of M0, first: {early[0]}"
