"""Registers of the microscaled 4-bit operators' kernels, read from the compiled
gfx950 code: a spill would wait for all loads on their way whenever it is read
back, which no parity test notices (no GPU needed)."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

from weight_only_quantization_quantize_amd import build as woq_build

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")

# source file -> the kernels it must hold, instances of each
FILES = {
    "mxfp4_quantize.hip": ["mxfp4_quantize_kernel", "mxfp4_dequantize_kernel", "mxfp4_split_kernel", "mxfp4_scales_kernel"],
    "mxfp4_gemv.hip": ["mxfp4_gemv_kernel"],
    "mxfp4_skinny.hip": ["mxfp4_skinny_kernel", "mxfp4_skinny_long_kernel"],
    "mxfp4_gemm.hip": ["mxfp4_gemm_kernel"],
    "mxfp4_moe.hip": ["moe_route_kernel", "moe_choose_kernel", "moe_experts_kernel", "moe_direct_down_kernel",
                      "moe_combine_kernel"],
}


@pytest.mark.parametrize("src", sorted(FILES))
def test_kernels_do_not_spill(src, tmp_path):
    out = str(tmp_path / "k.s")
    cmd = [HIPCC, "-x", "hip", *woq_build.COMMON_FLAGS, "--cuda-device-only", "-S", os.path.join(woq_build.CSRC, src), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    private = {}
    for m in re.finditer(r"\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", open(out).read(), re.S):
        private[m.group(1)] = int(re.search(r"\.amdhsa_private_segment_fixed_size (\d+)", m.group(2)).group(1))
    for name in FILES[src]:
        assert any(name in k for k in private), f"no {name} in {src}"
    spilling = {k: n for k, n in private.items() if n}
    assert not spilling, spilling
