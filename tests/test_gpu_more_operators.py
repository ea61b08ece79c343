"""The plain forms of the 8-bit operators compute the definition's scales and codes, so that
they say whether a kernel's outputs are right."""
import pytest
import torch

from perf import more_operators as plain
from tests.ffn_util import gen, normal
from tests.test_gpu_i8 import quant_ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
def test_plain_scales_and_codes(t):
    """Of 4096 rows, max |x| times the rounded 1/127 would miss the rounded quotient in some
    200."""
    x = normal(gen(1), (4096, 512), 1.0, t)
    q, s = quant_ref(x, 1)
    codes, scales = plain._quant(x.float(), 1)
    assert torch.equal(scales, s)
    assert torch.equal(codes, q)
