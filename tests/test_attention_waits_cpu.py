"""Every barrier of the prompt attention kernel waits for the loads into LDS before it (CPU; needs
hipcc): the tiles are loaded straight into LDS, so a wave must have waited (s_waitcnt vmcnt(0)) for
its own loads before the barrier after which the others read them.  Checked on the gfx950 assembly,
in straight-line order."""

import os
import re
import shutil
import subprocess

import pytest

from w4a16_dequant_gemm_amd import build

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def test_barriers_wait_for_the_tiles(tmp_path):
    if not os.path.exists(HIPCC) and shutil.which("hipcc") is None:
        pytest.skip("hipcc not available")
    out = tmp_path / "attention.s"
    cmd = [HIPCC, *build.HIPCC_FLAGS, "-x", "hip", "-S", "--cuda-device-only",
           os.path.join(build.CSRC, "attention.hip"), "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    kernels = re.findall(r"^(_ZN\S*attention_prompt_kernel\S*):\s*; @.*?$(.*?)^\.Lfunc_end", out.read_text(), re.M | re.S)
    assert len(kernels) == 8
    for name, body in kernels:
        loads = barriers = 0
        pending = False
        for line in body.splitlines():
            if re.search(r"\bbuffer_load_dwordx4\b.*\blds\b", line):
                loads += 1
                pending = True
            elif re.search(r"s_waitcnt.*vmcnt\(0\)", line):
                pending = False
            elif re.search(r"\bs_barrier\b", line):
                barriers += 1
                assert not pending, f"{name}: a barrier follows loads into LDS without a wait"
        assert loads > 0 and barriers > 0, name
