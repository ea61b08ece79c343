"""The 8-bit products load LDS through inline asm as the feed-forward block's do: the same
scan of their compiled kernels."""
import shutil

import pytest

from tests.test_ffn_asm_hazards import HIPCC, test_ffn_kernels_have_no_valu_sgpr_hazard as scan


@pytest.mark.skipif(shutil.which(HIPCC) is None, reason="hipcc not available")
def test_i8_kernels_have_no_valu_sgpr_hazard(tmp_path):
    scan(tmp_path, "i8.hip")
