"""The dense feed-forward block's kernels load LDS through inline asm as the MoE
layer's do: the same scan for buffer descriptors that a VALU op wrote too few wait
states before such a load."""
import os
import re
import shutil
import subprocess

import pytest

from sparse_expert_ffn_amd import buildlib
from tests.test_asm_hazards import lds_load_hazards

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.mark.skipif(shutil.which(HIPCC) is None, reason="hipcc not available")
@pytest.mark.parametrize("source", ["ffn_forward.hip", "ffn_backward.hip"])
def test_ffn_kernels_have_no_valu_sgpr_hazard(tmp_path, source):
    csrc = os.path.join(buildlib.PKG, "csrc")
    out = tmp_path / "kernels.s"
    flags = [f for f in buildlib.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    cmd = [HIPCC, *flags, "-I", os.path.join(buildlib.ROOT, "include"), "-I", csrc, "-I",
           os.path.join(csrc, "ffn"), "-S", "--cuda-device-only",
           os.path.join(csrc, "ffn", source), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    asm = out.read_text()
    assert re.search(r"\slds\b", asm), "no LDS-direct loads found in the assembly"
    found = lds_load_hazards(asm)
    assert not found, "\n".join(f"{k}: {w} wait states before {t}" for k, w, t in found[:10])
    # no kernel spills: a spill's memory traffic would count in the loads' vmcnt waits
    assert not re.search(r"\.vgpr_spill_count:\s*[1-9]", asm)
    assert not re.search(r"ScratchSize: [1-9]", asm)
