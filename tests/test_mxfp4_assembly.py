"""Inline assembly of the microscaled operators' kernels, read from the compiler's
intermediate code (no GPU needed): a statement that writes M0 says so, since the
compiler may keep a value of its own there."""
from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess

import pytest

from weight_only_quantization_quantize_amd import build as woq_build

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
WRITES_M0 = re.compile(r"\bs_\w+ m0,")
SOURCES = [f for f in sorted(glob.glob(os.path.join(woq_build.CSRC, "*.hip"))) if WRITES_M0.search(open(f).read())]


def test_some_source_writes_m0():
    assert SOURCES


@pytest.mark.parametrize("src", SOURCES, ids=os.path.basename)
def test_assembly_declares_its_write_of_m0(src, tmp_path):
    out = str(tmp_path / "k.ll")
    cmd = [HIPCC, "-x", "hip", *woq_build.COMMON_FLAGS, "--cuda-device-only", "-S", "-emit-llvm", src, "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    found = 0
    for text, constraints in re.findall(r'asm sideeffect "([^"]*)", "([^"]*)"', open(out).read()):
        if WRITES_M0.search(text):
            found += 1
            assert "~{m0}" in constraints.split(","), (text, constraints)
    assert found
