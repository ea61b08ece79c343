"""Layer norm, forward and backward, against 64-bit forms with derived bounds."""
import pytest
import torch

import sparse_expert_ffn_amd as moe
from sparse_expert_ffn_amd.layer import LayerNormBuffers
from tests.ffn_util import DEV, check, gen, half, ln_bwd_ref, ln_ref, normal

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
MD = {BF: moe.MOE_BF16, F32: moe.MOE_F32}

# one element, less than a vector, odd lengths, the edges of the wave and workgroup
# kernels (bf16: 2048, 16384; fp32: 1024, 8192; element-wise: 512, 4096), longer rows
SHAPES = [(1, 1), (5, 3), (64, 8), (3, 40), (7, 511), (9, 512), (4, 513), (130, 1001),
          (33, 1024), (6, 1032), (17, 2048), (5, 2056), (3, 4097), (2, 8192), (3, 8200),
          (2, 16384), (3, 16392), (2, 20001), (1, 65544), (3000, 72), (1025, 264),
          # each number of vectors or elements per thread in between
          (9, 101), (9, 201), (6, 301), (5, 701), (4, 1501), (4, 2501), (3, 5001), (3, 3600),
          (3, 5000), (3, 6200), (2, 9600), (2, 12800),
          # rows that end inside a vector, of every kernel; rows shorter than a vector;
          # groups of several rows
          (3, 3601), (3, 7001), (2, 9001), (2, 13001), (40, 5), (300, 2), (5000, 7), (9, 65),
          (2000, 33), (9, 129), (9, 257), (700, 2049), (600, 1003), (2100, 520), (530, 9001)]


def make(S, H, t, seed):
    g = gen(seed)
    off = torch.randn(H, generator=g, device=DEV) * 2
    x = (torch.randn((S, H), generator=g, device=DEV) + off).to(t)
    return x, normal(g, (H,), 0.2, t, 1.0), normal(g, (H,), 0.3, t), normal(g, (S, H), 0.5, t)


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("S,H", SHAPES)
def test_forward_and_backward(S, H, t):
    print(f"[layernorm {S}x{H} {t}]", flush=True)
    x, gamma, beta, dy = make(S, H, t, 1)
    b = LayerNormBuffers(S, H, MD[t], device=DEV)
    b.ws.fill_(0xFF)
    y = b.forward(x, gamma, beta, eps=1e-5)
    ry, rm, rr, ey, em, er = ln_ref(x, gamma, beta, 1e-5)
    check("mean", b.mean, rm, em)
    check("rstd", b.rstd, rr, er)
    check("y", y, ry, ey + half(t) * (ry.abs() + ey) + 1e-38)
    dx, dg, db = b.backward(dy, x, gamma)
    rx, rg, rb, ex, eg, eb = ln_bwd_ref(dy, x, gamma, b.mean, b.rstd)
    check("dx", dx, rx, ex + half(t) * (rx.abs() + ex) + 1e-38)
    check("dgamma", dg, rg, eg)
    check("dbeta", db, rb, eb)
    first = [v.clone() for v in (dx, dg, db)]
    b.backward(dy, x, gamma)
    assert all(torch.equal(p, q) for p, q in zip(first, (dx, dg, db))), "not reproducible"


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
def test_without_weights_and_statistics(t):
    x, _, _, dy = make(50, 264, t, 2)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    moe.moe_layernorm_forward(x, None, None, 1e-3, y)
    ry, rm, rr, ey, _, _ = ln_ref(x, None, None, 1e-3)
    check("y", y, ry, ey + half(t) * (ry.abs() + ey))
    mean, rstd = rm.float(), rr.float()
    moe.moe_layernorm_backward(dy, x, None, mean, rstd, dx, None, None, None)
    rx, _, _, ex, _, _ = ln_bwd_ref(dy, x, None, mean, rstd)
    check("dx", dx, rx, ex + half(t) * (rx.abs() + ex))


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", [64, 2056, 20000])
def test_arrays_off_16_bytes(t, H):
    """Bases that only an element's alignment holds for give the vector path's values."""
    S = 5
    x, gamma, beta, dy = make(S, H, t, 3)

    def shifted(v):
        s = torch.empty(v.numel() + 1, dtype=v.dtype, device=DEV)[1:].view(v.shape)
        return s.copy_(v)

    y = shifted(torch.zeros_like(x))
    mean, rstd = torch.empty(S, device=DEV), torch.empty(S, device=DEV)
    moe.moe_layernorm_forward(shifted(x), shifted(gamma), shifted(beta), 1e-5, y, mean, rstd)
    ry, rm, rr, ey, em, er = ln_ref(x, gamma, beta, 1e-5)
    check("y", y, ry, ey + half(t) * (ry.abs() + ey))
    dx = shifted(torch.zeros_like(x))
    dg, db = torch.empty(H, device=DEV), torch.empty(H, device=DEV)
    ws = torch.empty(moe.moe_layernorm_backward_workspace_bytes(S, H, MD[t]), dtype=torch.uint8,
                     device=DEV)
    moe.moe_layernorm_backward(shifted(dy), shifted(x), shifted(gamma), mean, rstd, dx, dg, db,
                               ws)
    rx, rg, rb, ex, eg, eb = ln_bwd_ref(dy, x, gamma, mean, rstd)
    check("dx", dx, rx, ex + half(t) * (rx.abs() + ex))
    check("dgamma", dg, rg, eg)
    check("dbeta", db, rb, eb)


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("S,H", [(1, 1), (3, 3), (37, 7), (5, 33), (130, 130), (6, 511), (3, 2049),
                                 (2, 9001), (2, 20001), (3, 64), (600, 1000)])
def test_nothing_beside_the_outputs_is_written(S, H, t):
    x, gamma, beta, dy = make(S, H, t, 6)
    n = moe.moe_layernorm_backward_workspace_bytes(S, H, MD[t])
    pad = 64  # elements or bytes on either side

    def framed(shape, dtype):
        size = int(torch.tensor(shape).prod())
        b = torch.full((size + 2 * pad,), 7, dtype=dtype, device=DEV)
        return b, b[pad:pad + size].view(shape)

    out = [framed((S, H), t), framed((S,), F32), framed((S,), F32), framed((S, H), t),
           framed((H,), F32), framed((H,), F32), framed((n,), torch.uint8)]
    y, mean, rstd, dx, dg, db, ws = (v for _, v in out)
    moe.moe_layernorm_forward(x, gamma, beta, 1e-5, y, mean, rstd)
    moe.moe_layernorm_backward(dy, x, gamma, mean, rstd, dx, dg, db, ws)
    for b, _ in out:
        assert bool((b[:pad] == 7).all()) and bool((b[-pad:] == 7).all())


def test_large_offset_keeps_the_variance():
    """Rows of 4096 + noise: the squares are centred before they are summed."""
    g = gen(4)
    x = torch.randn((8, 1024), generator=g, device=DEV) * 0.5 + 4096
    y = torch.empty_like(x)
    moe.moe_layernorm_forward(x, None, None, 0.0, y)
    ry, _, _, ey, _, _ = ln_ref(x, None, None, 0.0)
    check("y", y, ry, ey + half(F32) * ry.abs())
    assert float(ey.max()) < 0.1  # the bound says something


def test_constant_rows_and_not_finite_rows():
    x = torch.ones((4, 512), device=DEV)
    x[1, 7] = float("inf")
    x[2, 0] = float("nan")
    y = torch.empty_like(x)
    moe.moe_layernorm_forward(x, None, None, 1e-5, y)
    assert torch.equal(y[0], torch.zeros(512, device=DEV)) and torch.equal(y[3], y[0])
    assert bool(torch.isnan(y[1]).any()) and bool(torch.isnan(y[2]).all())


def test_no_rows():
    for t in (BF, F32):
        x = torch.empty((0, 64), dtype=t, device=DEV)
        b = LayerNormBuffers(0, 64, MD[t], device=DEV)
        b.dgamma.fill_(7)
        b.dbeta.fill_(7)
        b.forward(x)
        b.backward(x, x)
        assert float(b.dgamma.abs().max()) == 0 and float(b.dbeta.abs().max()) == 0


def test_gradient_against_differences():
    """Along a random direction v: (L(x + e v) - L(x - e v)) / 2 e = <dx, v> for L =
    sum c y, the differences taken in 64 bits."""
    g = gen(5)
    S, H = 6, 96
    x = torch.randn((S, H), generator=g, device=DEV)
    gamma = torch.randn(H, generator=g, device=DEV)
    c = torch.randn((S, H), generator=g, device=DEV)
    v = torch.randn((S, H), generator=g, device=DEV).double()
    b = LayerNormBuffers(S, H, moe.MOE_F32, device=DEV)
    b.forward(x, gamma)
    dx, dg, db = b.backward(c, x, gamma)

    def loss(z, gm):
        m = z.mean(1, keepdim=True)
        return float((c.double() * ((z - m) / ((z - m).square().mean(1, keepdim=True) + 1e-5)
                                    .sqrt() * gm)).sum())

    e = 1e-4  # the difference's own error is e^2 = 1e-8 of third derivatives of order 10
    num = (loss(x.double() + e * v, gamma.double()) - loss(x.double() - e * v, gamma.double())) \
        / (2 * e)
    assert abs(num - float((dx.double() * v).sum())) < 1e-4
    w = v[0]
    num = (loss(x.double(), gamma.double() + e * w) - loss(x.double(), gamma.double() - e * w)) \
        / (2 * e)
    assert abs(num - float((dg.double() * w).sum())) < 1e-4


@pytest.mark.timeout(300)
@pytest.mark.parametrize("H", [(1 << 27) - 1, (1 << 27) - 8])
def test_longest_rows(H):
    """The ends of the documented range, where one workgroup for each 64 column sums would
    be a launch of 2^32 threads."""
    print(f"[layernorm 1x{H}]", flush=True)
    x, gamma, _, dy = make(1, H, BF, 7)
    mean, rstd = torch.tensor([0.1], device=DEV), torch.tensor([0.5], device=DEV)
    dx, dg, db = torch.empty_like(x), torch.empty(H, device=DEV), torch.empty(H, device=DEV)
    ws = torch.empty(moe.moe_layernorm_backward_workspace_bytes(1, H), dtype=torch.uint8,
                     device=DEV)
    moe.moe_layernorm_backward(dy, x, gamma, mean, rstd, dx, dg, db, ws)
    n = (x[0].double() - mean.double()) * rstd.double()
    # one row: no sums; x - mean, its product with rstd and with dy are rounded
    check("dgamma", dg, dy[0].double() * n, 4 * 2.0 ** -24 * (dy[0].double() * n).abs() + 1e-38)
    assert torch.equal(db, dy[0].float())


@pytest.mark.timeout(300)
@pytest.mark.parametrize("H", [1 << 24, (1 << 24) + 3, 1 << 26])
def test_long_rows_of_nearly_equal_values(H):
    """Each of the sums over a row is within 20 roundings of its terms' magnitudes, however
    long the row: 3 within a vector, 2 of the compensated sum over vectors, 6 within the
    wave and 3 over the waves, 4 for the terms themselves, 2 for the division by H."""
    print(f"[layernorm 1x{H}]", flush=True)
    g = gen(8)
    x = (torch.randn((1, H), generator=g, device=DEV) * 1e-3 + 0.1)
    dy = (torch.randn((1, H), generator=g, device=DEV) * 1e-3 + 0.1)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    moe.moe_layernorm_forward(x, None, None, 1e-9, y, mean, rstd)
    u, k = 2.0 ** -24, 20
    x64 = x.double()
    m = x64.mean()
    v = (x64 - m).square().mean()
    r = 1 / torch.sqrt(v + 1e-9)
    em = k * u * x64.abs().mean()
    er = r * (0.5 * (k * u * v + em * em) / (v + 1e-9) + 4 * u)  # cf. ln_ref
    check("mean", mean, m[None], em[None])
    check("rstd", rstd, r[None], er[None])
    n = (x64 - m) * r
    check("y", y, n, r * em + n.abs() * (er / r + 5 * u))
    moe.moe_layernorm_backward(dy, x, None, mean, rstd, dx, None, None, None)
    n = (x64 - mean.double()) * rstd.double()
    d = dy.double()
    c0, c1 = d.mean(), (d * n).mean()
    e0, e1 = k * u * d.abs().mean(), k * u * (d * n).abs().mean()
    check("dx", dx, rstd.double() * (d - c0 - n * c1),
          rstd.double() * (e0 + n.abs() * e1 + 6 * u * (d.abs() + c0.abs() + (n * c1).abs())))


def test_long_rows_that_are_not_finite():
    """A sum that leaves fp32's range, and infinities and NaN, as in shorter rows."""
    H = 20008
    x = torch.ones((5, H), device=DEV)
    x[1, 7], x[2, 9], x[3, 11] = float("inf"), float("-inf"), float("nan")
    x[4] = 3e38
    y = torch.empty_like(x)
    mean, rstd = torch.empty(5, device=DEV), torch.empty(5, device=DEV)
    moe.moe_layernorm_forward(x, None, None, 1e-5, y, mean, rstd)
    inf = float("inf")
    assert mean[:3].tolist() == [1.0, inf, -inf] and bool(torch.isnan(mean[3]))
    assert float(mean[4]) == inf and bool((y[0] == 0).all())
    assert bool(torch.isnan(y[1, 7])) and bool(torch.isnan(y[3]).all())
