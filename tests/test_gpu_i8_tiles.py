"""8-bit products and blocks at sizes that take every tile, with K whole and split, weights read
once or more often, and every way from h to its codes (tests/test_i8_plan.py holds what each
case takes)."""
import pytest
import torch

import sparse_expert_ffn_amd as moe
from sparse_expert_ffn_amd.layer import I8Weight
from tests.ffn_util import DEV, check, gen, half, normal
from tests.test_gpu_i8 import ffn_ref, product, quant_ref, weight
from tests.test_i8_plan import FFN, MATMUL

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def guarded(S, N, t):
    """[S][N] of NaN with rows behind it that have to stay."""
    full = torch.full((S + 2, N), float("nan"), dtype=t, device=DEV)
    full[S:] = 7.0
    return full, full[:S]


def workspace(n):
    """n bytes of 0xFF with 64 behind them that have to stay."""
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    ws[n:] = 0x35
    return ws, ws[:n]


@pytest.mark.parametrize("S,K,N", list(MATMUL))
def test_matmul(S, K, N):
    print(f"[matmul {S}x{K}x{N}]", flush=True)
    g = gen(30)
    x, w = normal(g, (S, K), 1.0, BF), weight(g, K, N)
    q, s = quant_ref(x, 1)
    ref, e = product(q, s[:, 0], w)
    wt = I8Weight(*w)
    n = moe.moe_i8_matmul_workspace_bytes(S, K, N)
    for t in (F32, BF):
        full, y = guarded(S, N, t)
        ws_full, ws = workspace(n)
        moe.moe_i8_matmul(x, wt, y, ws)
        check("y", y, ref, e + half(t) * (ref.abs() + e) + 1e-38)
        assert bool((full[S:] == 7.0).all()) and bool((ws_full[n:] == 0x35).all())


@pytest.mark.parametrize("S,H,D", list(FFN))
def test_ffn(S, H, D):
    print(f"[ffn {S}x{H}x{D}]", flush=True)
    g = gen(31)
    x = normal(g, (S, H), 1.0, BF)
    w = weight(g, H, D), weight(g, H, D), weight(g, D, H)
    ref, e = ffn_ref(x, *w)
    wt = [I8Weight(*v) for v in w]
    for t in (F32, BF):
        shape = moe.make_ffn_shape(S, H, D, out_f32=t == F32)
        n = moe.moe_i8_ffn_workspace_bytes(shape)
        full, o = guarded(S, H, t)
        ws_full, ws = workspace(n)
        moe.moe_i8_ffn_forward(shape, x, *wt, o, ws)
        check("o", o, ref, e + half(t) * (ref.abs() + e))
        assert bool((full[S:] == 7.0).all()) and bool((ws_full[n:] == 0x35).all())
