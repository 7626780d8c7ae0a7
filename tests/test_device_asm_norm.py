"""The gfx950 assembly of the norms' kernels (CPU only): no packed fp32 arithmetic, and no more
registers spilled than stated. Where a row and its sums leave no register free a few are; beyond
that the traffic of the spills reaches that of the row."""
import os
import re
import shutil
import subprocess

import pytest

from rank_randomized_gradient_amd import build


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    cc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(cc):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("norm") / "out.s"
    flags = [f for f in build.HIP_FLAGS if f not in ("-fPIC", "-Wall", "-Wno-unused-function")]
    cmd = [cc, *flags, "--cuda-device-only", "-S", os.path.join(build.CSRC, "rgc_norm.hip"), "-o", str(out)]
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert res.returncode == 0, res.stdout[-2000:]
    return out.read_text()


def test_no_packed_fp32(asm):
    assert not re.findall(r"v_pk_(?:add|mul|fma)_f32", asm)


def test_spills(asm):
    """By kernel: type, vectors of a thread, threads of a row and of a workgroup, residual (and the bias's gradient)."""
    spills = {}
    for block in asm[asm.index("amdhsa.kernels"):asm.index("amdhsa.target")].split("\n  - ")[1:]:
        name = re.search(r"^    \.name:\s+(\S+)", block, re.M).group(1)
        spills[name] = int(re.search(r"\.vgpr_spill_count:\s+(\d+)", block).group(1))
    seen = {"forward": 0, "backward": 0}
    for name, count in spills.items():
        m = re.search(r"norm_(forward|backward)_kernelI([tf])Lb([01])ELi(\d+)ELi(\d+)ELi(\d+)ELb([01])E(?:Lb([01])E)?E", name)
        if not m:
            assert count == 0, name
            continue
        which, vectors, threads, add, db = m.group(1), int(m.group(4)), int(m.group(6)), m.group(7) == "1", m.group(8) == "1"
        seen[which] += 1
        if which == "forward":
            # rows above 16384: eight vectors in the 128 registers of 1024 threads
            most = 64 if vectors == 8 and threads == 1024 else 0
        elif add and db:
            most = 16 if vectors == 8 else 0  # bf16: three rows' vectors and two rows' sums in 256
        else:
            most = 8 if vectors == 4 and threads == 1024 else 0
        assert count <= most, (name, count)
    assert seen["forward"] >= 40 and seen["backward"] >= 40, seen
