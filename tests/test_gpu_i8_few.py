"""8-bit products of few rows: what the one-launch form's workgroups do for themselves (rows
quantised by one or several waves, in one or more rounds, longer than a thread keeps), and that
it gives the bits of the tiles', wherever it gives way to them."""
import pytest
import torch

import sparse_expert_ffn_amd as moe
from sparse_expert_ffn_amd.layer import I8LinearBuffers, I8Weight
from tests.ffn_util import DEV, check, gen, half, normal
from tests.test_gpu_i8 import awkward, product, quant_ref, weight

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("S,K,N", [(1, 64, 24), (1, 48, 5128), (3, 8208, 40), (5, 16400, 72),
                                   (8, 4096, 16), (9, 208, 264), (16, 1040, 40), (16, 8176, 24),
                                   (1, 130000, 16), (16, 8192, 24), (11, 80, 16392)])
def test_few_rows(S, K, N, t):
    """With rows of zeros, tiny, huge and non-finite values. The last two of the few rows are
    past the one-launch form's limits."""
    print(f"[few rows {S}x{K}x{N}]", flush=True)
    g = gen(20)
    x, w = awkward(normal(g, (S, K), 1.0, t)), weight(g, K, N)
    if S > 5:
        x[5] *= 1e-3  # 3e38 times a sum of codes is past fp32
    q, s = quant_ref(x, 1)
    ref, e = product(q, torch.nan_to_num(s[:, 0], 0.0), w)
    b = I8LinearBuffers(S, K, N, dtype=moe.MOE_F32 if t == F32 else moe.MOE_BF16, out_f32=True,
                        device=DEV)
    b.Y.fill_(7.0)
    b.run(x, I8Weight(*w))
    bad = torch.isnan(s[:, 0])
    assert bool(torch.isnan(b.Y[bad]).all()) and int(bad.sum()) == (2 if S > 8 else 0)
    check("y", b.Y[~bad], ref[~bad], e[~bad] + half(F32) * ref[~bad].abs() + 1e-38)


@pytest.mark.parametrize("K,N", [(528, 72), (2064, 264)])
def test_one_row_alone_and_among_many(K, N):
    """A row's bits do not depend on how many others there are."""
    g = gen(21)
    x, w = normal(g, (300, K), 1.0, BF), I8Weight(*weight(g, K, N))
    many = I8LinearBuffers(300, K, N, device=DEV).run(x, w)
    for S in (1, 2, 7, 16, 17, 40):
        b = I8LinearBuffers(S, K, N, device=DEV)
        assert torch.equal(b.run(x[10:10 + S].contiguous(), w), many[10:10 + S]), S
