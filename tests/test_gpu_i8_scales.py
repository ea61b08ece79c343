"""Scales that the library's own quantisation does not give: signs, and magnitudes whose
product with a sum of codes is past fp32 before the other scale brings it back."""
import pytest
import torch

from sparse_expert_ffn_amd.layer import FewMoEBuffers, I8LinearBuffers, I8Weight
from tests.ffn_util import DEV, check, gen, half
from tests.test_gpu_i8 import product

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("S", [1, 16, 40, 300])
def test_signed_scales(S):
    """Every pair of signs, the larger magnitude on either side; sums up to 2 x 10^8."""
    g = gen(60)
    K, N = 16384, 72
    q = torch.randint(100, 128, (S, K), generator=g, device=DEV, dtype=torch.int8)
    codes = torch.randint(100, 128, (K, N), generator=g, device=DEV, dtype=torch.int8)
    for a, b in ((1e-30, 1e31), (1e31, 1e-30), (0.5, 0.25)):
        s = a * (1 + torch.rand(S, generator=g, device=DEV))
        w = b * (1 + torch.rand(N, generator=g, device=DEV))
        s[1::2] *= -1
        w[1::3] *= -1
        y = I8LinearBuffers(S, K, N, out_f32=True, device=DEV)
        y.run(q, I8Weight(codes, w), row_scales=s)
        ref, e = product(q, s, (codes, w))
        check(f"{a} {b}", y.Y, ref, e + half(F32) * (ref.abs() + e))


def test_signed_scales_of_experts():
    """The layer with codes and scales negated is the layer: h's two factors and y change their
    signs together."""
    g = gen(61)
    S, H, D, E, k = 5, 272, 144, 8, 2
    w = [(torch.randint(-127, 128, (E, K, N), generator=g, device=DEV, dtype=torch.int8),
          (torch.rand((E, N), generator=g, device=DEV) + 0.5) / (74 * K ** 0.5))
         for K, N in ((H, D), (H, D), (D, H))]
    x = torch.randn((S, H), generator=g, device=DEV).to(BF)
    wr = (0.1 * torch.randn((H, E), generator=g, device=DEV)).to(BF)
    a, b = (FewMoEBuffers(S, H, D, E, k, i8=True, device=DEV) for _ in range(2))
    a.run(x, wr, *(I8Weight(q, s) for q, s in w))
    b.run(x, wr, *(I8Weight(-q, -s) for q, s in w))
    assert torch.equal(a.O, b.O)
