"""The accumulated weights may be added up in place (`sums` is `weights`): no kernel that takes both may tell
the compiler that they differ (CPU; needs hipcc).  Checked on the kernels' parameters in the gfx950 IR."""

import os
import re
import shutil
import subprocess

import pytest

from w4a16_dequant_gemm_amd import build

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def test_weights_and_sums_may_be_one(tmp_path):
    if not os.path.exists(HIPCC) and shutil.which("hipcc") is None:
        pytest.skip("hipcc not available")
    out = tmp_path / "kv_attend.ll"
    cmd = [HIPCC, *build.HIPCC_FLAGS, "-x", "hip", "-S", "-emit-llvm", "--cuda-device-only",
           os.path.join(build.CSRC, "kv_attend.hip"), "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    found = 0
    for name, params in re.findall(r"^define .*amdgpu_kernel void @(_ZN\S*kv_(?:weights|whole)_kernel\S*?)\((.*)\) [^()]*\{$",
                                   out.read_text(), re.M):
        mine = re.split(r", (?=ptr|i\d)", params)[-2:]          # weights, sums
        assert len(mine) == 2 and all(p.startswith("ptr") for p in mine), f"{name}: {mine}"
        found += 1
        assert not any("noalias" in p for p in mine), f"{name}: {mine}"
    assert found >= 2 + 4 * 3                   # D = 64 / 128; both code widths, three ways to keep scores
