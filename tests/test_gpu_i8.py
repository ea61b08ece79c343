"""8-bit integers with a scale per token and channel: quantisation and packing exactly,
products and the gated block against 64-bit forms."""
import pytest
import torch

import sparse_expert_ffn_amd as moe
from sparse_expert_ffn_amd.layer import I8FFNBuffers, I8LinearBuffers, I8Weight
from tests.ffn_util import DEV, U, check, gen, half, mm, normal

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def quant_ref(x, dim):
    """Codes and scales by the formula; the quotient in 64 bits decides exactly (two fp32
    numbers whose quotient is no half integer are further from one than 2^-53)."""
    x = x.cpu()
    top = x.float().abs().amax(dim, keepdim=True)
    s = (top.double() / 127).float()  # rounded once: a quotient of fp32 numbers in 64 bits
    live = (s > 0) & torch.isfinite(top)
    q = torch.round(torch.where(live, x.double() / torch.where(live, s, 1.0).double(), 0.0))
    s = torch.where(torch.isfinite(x).all(dim, keepdim=True), s, float("nan"))
    return q.clamp(-127, 127).to(torch.int8).to(DEV), s.to(DEV)


def same(a, b):
    return torch.equal(torch.nan_to_num(a, 7e30), torch.nan_to_num(b, 7e30))


def awkward(x):
    """Rows (few as there may be) with zeros, tiny, huge and non-finite values, borders
    between codes, one large value."""
    S, K = x.shape
    rows = [torch.zeros(K), torch.full((K,), 2.0 ** -133), torch.arange(K) % 255 - 127.0,
            (torch.arange(K) % 255 - 127.0) / 2, torch.full((K,), 1e-30), torch.full((K,), 3e38)]
    for i, r in enumerate(rows):
        if i < S:
            x[i] = r.to(x)
    if S > 6:
        x[5, 3] = 254.0
    if S > 8:
        x[6, K - 1], x[7, 0] = float("nan"), float("-inf")
        x[8, 1] = 1e30
    return x


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("S,K", [(1, 16), (3, 48), (9, 2048), (70, 4096), (11, 4112), (9, 7168),
                                 (10, 16384), (10, 16400), (9, 65552), (9, 131072)])
def test_quantize_rows(S, K, t):
    print(f"[rows {S}x{K}]", flush=True)
    x = awkward(normal(gen(1), (S, K), 1.0, t))
    codes = torch.full((S, K), 99, dtype=torch.int8, device=DEV)
    scales = torch.full((S,), 5.0, device=DEV)
    moe.moe_quantize_i8_rows(x, codes, scales)
    q, s = quant_ref(x, 1)
    assert same(scales, s[:, 0])
    assert torch.equal(codes, q), (codes != q).nonzero()[:5]


def test_quantize_rows_borders():
    """Quotients that lie on a border between two codes, or next to it by an ulp of x."""
    g = gen(2)
    S, K = 512, 1024
    top = torch.rand((S, 1), generator=g, device=DEV) + 0.5
    top[:100] = torch.randint(1, 128, (100, 1), generator=g, device=DEV) / 8.0
    n = torch.randint(-126, 126, (S, K), generator=g, device=DEV) + 0.5
    s = (top.double() / 127).float()
    x = (n.double() * s.double()).float()
    x[:, 1::3] = torch.nextafter(x[:, 1::3], torch.full_like(x[:, 1::3], 1e9))
    x[:, 2::3] = torch.nextafter(x[:, 2::3], torch.full_like(x[:, 2::3], -1e9))
    x[:, 0] = top[:, 0]
    codes = torch.empty((S, K), dtype=torch.int8, device=DEV)
    scales = torch.empty(S, device=DEV)
    moe.moe_quantize_i8_rows(x, codes, scales)
    q, s = quant_ref(x, 1)
    assert same(scales, s[:, 0]) and torch.equal(codes, q)


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("E,K,N", [(1, 16, 8), (2, 80, 24), (3, 256, 136), (1, 1040, 264)])
def test_quantize_weights(E, K, N, t):
    w = awkward(normal(gen(3), (E * N, K), 0.3, t)).view(E, N, K).transpose(1, 2).contiguous()
    codes = torch.empty((E, K, N), dtype=torch.int8, device=DEV)
    scales = torch.empty((E, N), device=DEV)
    moe.moe_quantize_i8(w, codes, scales)
    q, s = quant_ref(w, 1)
    assert same(scales, s[:, 0]) and torch.equal(codes, q)


@pytest.mark.parametrize("E,K,N", [(1, 64, 16), (2, 80, 24), (1, 144, 136)])
def test_packed_layout(E, K, N):
    """Byte by byte as the header describes it."""
    g = gen(4)
    codes = torch.randint(-128, 128, (E, K, N), generator=g, device=DEV, dtype=torch.int8)
    scales = torch.rand((E, N), generator=g, device=DEV)
    p = I8Weight(codes, scales).packed.cpu()
    nt, kt = -(-N // 16), -(-K // 64)
    size = nt * kt * 1024 + nt * 64
    assert p.numel() == E * size
    full = torch.zeros((E, kt * 64, nt * 16), dtype=torch.int8)
    full[:, :K, :N] = codes.cpu()
    fs = torch.zeros((E, nt * 16))
    fs[:, :N] = scales.cpu()
    # [E][kt][4 q][16 i][nt][16 c] -> [E][nt][kt][q][c][i]
    want = full.view(E, kt, 4, 16, nt, 16).permute(0, 4, 1, 2, 5, 3).reshape(E, -1)
    for e in range(E):
        m = p[e * size:(e + 1) * size]
        assert torch.equal(m[:nt * kt * 1024].view(torch.int8), want[e])
        assert torch.equal(m[nt * kt * 1024:].view(F32), fs[e])


def weight(g, K, N, E=None):
    shape = (K, N) if E is None else (E, K, N)
    codes = torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)
    scales = (torch.rand((*shape[:-2], N), generator=g, device=DEV) + 0.5) / (74 * K ** 0.5)
    return codes, scales


def product(q, s, w):
    """sum of codes' products (exact), scaled; and the bound before the output's rounding: the
    integer's rounding to fp32 and two products."""
    y = mm(q, w[0]) * s.double()[:, None] * w[1].double()
    return y, 3 * U * y.abs()


SIZES = [(1, 16, 8), (1, 7168, 64), (2, 144, 24), (3, 2064, 264), (15, 208, 72), (16, 1024, 128),
         (17, 272, 40), (33, 528, 136), (64, 128, 512), (70, 80, 200), (130, 1040, 392),
         (300, 336, 520), (257, 4112, 264), (1001, 192, 776), (1, 131072, 16)]


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("S,K,N", SIZES)
def test_matmul(S, K, N, t):
    print(f"[matmul {S}x{K}x{N}]", flush=True)
    g = gen(5)
    x, w = normal(g, (S, K), 1.0, t), weight(g, K, N)
    q, s = quant_ref(x, 1)
    ref, e = product(q, s[:, 0], w)
    wt = I8Weight(*w)
    for out_f32 in (False, True):
        b = I8LinearBuffers(S, K, N, dtype=moe.MOE_F32 if t == F32 else moe.MOE_BF16,
                            out_f32=out_f32, device=DEV)
        b.ws.fill_(0xFF)
        b.Y.fill_(float("nan"))
        b.run(x, wt)
        check("y", b.Y, ref, e + half(b.Y.dtype) * (ref.abs() + e) + 1e-38)
        y = b.Y.clone()
        b.Y.fill_(float("nan"))
        b.ws.fill_(0x7F)
        b.run(q, wt, row_scales=s[:, 0].contiguous())  # its codes give the same bits
        assert torch.equal(b.Y, y)


@pytest.mark.parametrize("S", [1, 20, 300])
def test_matmul_extreme_codes(S):
    """Every product of the largest magnitude, all of one sign: the sum next to 2^31."""
    K, N = 131072, 24
    q = torch.full((S, K), 127, dtype=torch.int8, device=DEV)
    w = torch.full((K, N), -128, dtype=torch.int8, device=DEV)
    w[:, 1::2] = 127
    b = I8LinearBuffers(S, K, N, out_f32=True, device=DEV)
    b.run(q, I8Weight(w, torch.ones(N, device=DEV)), row_scales=torch.ones(S, device=DEV))
    assert bool((b.Y[:, 0::2] == -127.0 * 128 * K).all())
    assert bool((b.Y[:, 1::2] == 127.0 * 127 * K).all())


@pytest.mark.parametrize("S", [3, 40, 300])
def test_matmul_rows_do_not_meet(S):
    """A row that holds a NaN or infinity gives a row of NaN and leaves the others."""
    g = gen(6)
    K, N = 528, 72
    x, w = normal(g, (S, K), 1.0, BF), I8Weight(*weight(g, K, N))
    b, c = (I8LinearBuffers(S, K, N, device=DEV) for _ in range(2))
    b.run(x, w)
    x2 = x.clone()
    x2[1, 100], x2[2, 5] = float("nan"), float("inf")
    c.run(x2, w)
    keep = torch.ones(S, dtype=torch.bool, device=DEV)
    keep[1] = keep[2] = False
    assert torch.equal(b.Y[keep], c.Y[keep]) and bool(torch.isnan(c.Y[1:3]).all())


def ffn_ref(x, up, gate, down):
    """(o, bound before rounding). u and g are exact integers scaled: off by 3 u each; exp and
    rcp by 2 u and the argument's error, so h by at most (12 + 4 |u|) u of itself. A code of
    h may move by one where h / s is that near to a border: 127 times its relative error on
    either side, a chance p <= 2 * 127 * (12 + 4 max |u|) u per value. Their number is
    binomial (an expected m <= D p, at most m + 6 sqrt(m) + 6 of them), each moves the output by
    one step of the row times the weight; six standard deviations of such a sum, with the
    largest weight of a column."""
    q, s = quant_ref(x, 1)
    (u, _), (g, _) = product(q, s[:, 0], up), product(q, s[:, 0], gate)
    h = u * torch.sigmoid(u) * g
    D = h.shape[1]
    top = h.abs().amax(1, keepdim=True)
    sh = (top / 127).float().double()
    qh = torch.where(sh > 0, torch.round(h / torch.where(sh > 0, sh, 1.0)), 0.0)
    wd = down[0].double() * down[1].double()
    o = mm(qh * sh, wd)
    eps = (12 + 4 * float(u.abs().max())) * U
    m = 2 * 127 * eps * D
    moved = min(m + 6 * m ** 0.5 + 6, D)
    e = sh * wd.abs().amax(0)[None] * min(moved, 6 * moved ** 0.5 + 6) + (eps + 5 * U) * o.abs()
    return o, e + 1e-38


@pytest.mark.parametrize("t,out_f32", [(BF, False), (BF, True), (F32, False)],
                         ids=["bf16", "bf16_f32", "f32"])
@pytest.mark.parametrize("S,H,D", [(1, 64, 80), (5, 272, 144), (16, 2048, 768), (33, 208, 400),
                                   (64, 512, 256), (130, 336, 208), (700, 256, 528)])
def test_ffn(S, H, D, t, out_f32):
    print(f"[ffn {S}x{H}x{D}]", flush=True)
    g = gen(7)
    x = normal(g, (S, H), 1.0, t)
    w = weight(g, H, D), weight(g, H, D), weight(g, D, H)
    if S > 3:
        x[2] = 0  # a row of zeros gives one
    o, e = ffn_ref(x, *w)
    b = I8FFNBuffers(S, H, D, dtype=moe.MOE_F32 if t == F32 else moe.MOE_BF16, out_f32=out_f32,
                     device=DEV)
    b.ws.fill_(0xFF)
    b.O.fill_(float("nan"))
    b.forward(x, *(I8Weight(*v) for v in w))
    check("o", b.O, o, e + half(b.O.dtype) * (o.abs() + e))
    if S > 3:
        assert not bool(b.O[2].any())


def test_ffn_is_its_products():
    """The block is the products and the activation between them, and reproducible."""
    g = gen(8)
    S, H, D = 40, 256, 144
    x = normal(g, (S, H), 1.0, BF)
    wu, wg, wd = (I8Weight(*v) for v in (weight(g, H, D), weight(g, H, D), weight(g, D, H)))
    b = I8FFNBuffers(S, H, D, device=DEV)
    o = b.forward(x, wu, wg, wd).clone()
    assert torch.equal(b.forward(x, wu, wg, wd), o)
    up, gate = (I8LinearBuffers(S, H, D, out_f32=True, device=DEV) for _ in range(2))
    u, v = up.run(x, wu), gate.run(x, wg)
    h = (u.double() * torch.sigmoid(u.double()) * v.double()).float()
    down = I8LinearBuffers(S, D, H, dtype=moe.MOE_F32, device=DEV)
    ref = down.run(h, wd).double()
    # h by way of 64 bits is off by its own rounding: at most some codes by one step
    step = h.double().abs().amax(1, keepdim=True) / 127
    wmax = 127 * wd.packed[-H * 4:].view(F32).double()
    check("o", o, ref, 6 * step * wmax[None] + half(BF) * (ref.abs() + 6 * step * wmax[None]))


def test_captured():
    """Product and block in one graph, replayed with other inputs and eager work between."""
    g = gen(9)
    S, H, D = 6, 256, 144
    x = normal(g, (S, H), 1.0, BF)
    wu, wg, wd = (I8Weight.quantize(normal(g, (K, N), K ** -0.5, BF))
                  for K, N in ((H, D), (H, D), (D, H)))
    mk = lambda: (I8LinearBuffers(S, H, D, device=DEV), I8FFNBuffers(S, H, D, device=DEV))
    (lin, ffn), (lin2, ffn2) = mk(), mk()
    step = lambda a, b: (a.run(x, wu), b.forward(x, wu, wg, wd))
    step(lin, ffn)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(lin, ffn)
    x0 = x.clone()
    for rep in range(4):
        x.copy_(x0 * (rep + 1))
        graph.replay()
        torch.cuda.synchronize()
        y, o = step(lin2, ffn2)
        assert torch.equal(lin.Y, y) and torch.equal(ffn.O, o), rep


def test_on_another_stream():
    g = gen(10)
    x, w = normal(g, (9, 512), 1.0, BF), weight(g, 512, 264)
    b, c = (I8LinearBuffers(9, 512, 264, device=DEV) for _ in range(2))
    b.run(x, I8Weight(*w))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    wt = I8Weight(*w, stream=side)
    c.run(x, wt, stream=side)
    c.Y.record_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(b.Y, c.Y)


def test_no_rows():
    w = I8Weight(*weight(gen(11), 64, 16))
    e = lambda *n, t=BF: torch.empty(n, dtype=t, device=DEV)
    moe.moe_i8_matmul(e(0, 64), w, e(0, 16), e(256, t=torch.uint8))
    moe.moe_quantize_i8_rows(e(0, 64), e(0, 64, t=torch.int8), e(0, t=F32))


def test_binding_refusals():
    w = I8Weight(*weight(gen(12), 64, 16))
    w2 = I8Weight(*weight(gen(12), 64, 16, E=2))
    e = lambda *n, t=BF: torch.zeros(n, dtype=t, device=DEV)
    x, y, ws = e(2, 64), e(2, 16), e(4096, t=torch.uint8)
    with pytest.raises(ValueError, match="W is"):
        moe.moe_i8_matmul(e(2, 32), w, y, ws)
    with pytest.raises(ValueError, match="W is"):
        moe.moe_i8_matmul(x, w2, y, ws)
    with pytest.raises(TypeError, match="I8Weight"):
        moe.moe_i8_matmul(x, x, y, ws)
    with pytest.raises(ValueError, match="Y is"):
        moe.moe_i8_matmul(e(2, 64, t=F32), w, y, ws)
    with pytest.raises(ValueError, match="X is"):
        moe.moe_i8_matmul(x, w, y, ws, row_scales=e(2, t=F32))
    with pytest.raises(ValueError, match="row_scales"):
        moe.moe_i8_matmul(e(2, 64, t=torch.int8), w, y, ws, row_scales=e(3, t=F32))
    with pytest.raises(moe.MoeError, match="WORKSPACE"):
        moe.moe_i8_matmul(x, w, y, ws[:16])
    with pytest.raises(ValueError, match="scales"):
        I8Weight(e(64, 16, t=torch.int8), e(1, 16, t=F32))
    with pytest.raises(moe.MoeError, match="UNSUPPORTED"):
        I8Weight(e(40, 16, t=torch.int8), e(16, t=F32))
    b = I8FFNBuffers(2, 64, 16, device=DEV)
    with pytest.raises(ValueError, match="W_down"):
        b.forward(x, w, w, w)
