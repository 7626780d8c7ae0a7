"""The gfx950 assembly of the clipping and of the logits' kernels (CPU only): no
packed fp32 arithmetic, no access through a flat address (what is shared in LDS is
read there), no register spilled."""
import os
import re
import shutil
import subprocess

import pytest

from rank_randomized_gradient_amd import build


@pytest.mark.parametrize("name", ["rgc_clip", "rgc_logits"])
def test_assembly(tmp_path, name):
    cc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(cc):
        pytest.skip("hipcc not available")
    out = tmp_path / "out.s"
    flags = [f for f in build.HIP_FLAGS if f not in ("-fPIC", "-Wall", "-Wno-unused-function")]
    cmd = [cc, *flags, "--cuda-device-only", "-S", os.path.join(build.CSRC, name + ".hip"), "-o", str(out)]
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert res.returncode == 0, res.stdout[-2000:]
    asm = out.read_text()
    assert not re.findall(r"v_pk_(?:add|mul|fma)_f32", asm)
    assert not re.findall(r"^\s*flat_(?:load|store|atomic)", asm, re.M)
    spills = [int(n) for n in re.findall(r"\.vgpr_spill_count:\s+(\d+)", asm)]
    assert spills and not any(spills)
