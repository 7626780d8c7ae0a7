"""The gfx950 assembly of the head's loss (CPU only): every global-to-LDS copy,
issued from inline asm, has its five wait states in front (as the other staged
kernels'), and the step loops of the large tile hold their sums in registers:
no scratch access and no move between register files among their MFMAs."""
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
    out = tmp_path_factory.mktemp("asm") / "loss.s"
    flags = [f for f in build.HIP_FLAGS if f not in ("-fPIC", "-Wall", "-Wno-unused-function")]
    cmd = [cc, *flags, "--cuda-device-only", "-S", os.path.join(build.CSRC, "rgc_loss.hip"), "-o", str(out)]
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert res.returncode == 0, res.stdout[-2000:]
    return out.read_text()


def test_every_lds_copy_has_five_wait_states(asm):
    prev, copies = None, 0
    for line in asm.split("\n"):
        s = line.strip()
        if not s or s.startswith((";", ".")) or s.endswith(":"):
            continue
        if s.startswith("global_load_lds"):
            copies += 1
            assert prev == "s_nop 4", f"{s} follows {prev}"
        prev = s
    assert copies > 0


def test_no_packed_fp32_arithmetic(asm):
    assert not re.findall(r"v_pk_(?:add|mul|fma)_f32", asm)


@pytest.mark.parametrize("kernel", ["ce_logits_kernelILb0ELb0", "ce_logits_kernelILb1ELb0", "ce_dx_kernel"])
def test_step_loops_stay_in_registers(asm, kernel):
    body = re.search(r"^_Z\S*%s\S*:(.*?)\n\.Lfunc_end" % kernel, asm, re.S | re.M).group(1)
    blocks = [b for b in re.split(r"\n\.LBB\S+:", body) if b.count("v_mfma") >= 48]
    assert blocks
    for b in blocks:
        assert "scratch_" not in b and "v_accvgpr" not in b
