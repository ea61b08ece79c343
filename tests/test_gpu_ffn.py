"""The dense gated feed-forward block, forward and backward, against 64-bit forms
with derived bounds."""
import pytest
import torch

import sparse_expert_ffn_amd as moe
from sparse_expert_ffn_amd.layer import FFNBuffers, LayerNormBuffers
from tests.ffn_util import DEV, check, ffn_bwd_ref, ffn_ref, gen, half, mm, normal

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
MD = {BF: moe.MOE_BF16, F32: moe.MOE_F32}

# one token, sizes below and off every tile, whole tiles, K shorter and longer than
# a stage, long K (splits), more rows than K
SHAPES = [(1, 8, 8), (1, 2048, 768), (3, 72, 40), (16, 64, 64), (17, 200, 136),
          (64, 128, 256), (65, 264, 520), (130, 2056, 72), (256, 256, 256), (257, 520, 1032),
          (300, 72, 2056), (1000, 256, 384), (2049, 64, 136), (100, 4096, 1024),
          (2048, 1024, 2048)]
# every tile of every product, with and without splits of K (the plan's choices at
# these sizes), whole and cut off in both directions
TILES = [(1, 1032, 2056), (1, 2056, 2056), (1, 2056, 4104), (17, 1032, 2056), (17, 2056, 1032),
         (60, 7168, 2056), (65, 2056, 4104), (65, 4104, 2056), (130, 1032, 2056), (130, 2056, 2056),
         (1025, 72, 2056), (1025, 136, 4104), (1025, 2056, 264), (1025, 4104, 72),
         (1025, 4104, 136), (1025, 4104, 2056), (2049, 72, 4104), (2049, 136, 72),
         (2049, 4104, 72), (4100, 72, 2056), (4100, 136, 2056), (4100, 2056, 72)]


def make(S, H, D, t, seed):
    g = gen(seed)
    return (normal(g, (S, H), 1.0, t), normal(g, (H, D), H ** -0.5, t),
            normal(g, (H, D), H ** -0.5, t), normal(g, (D, H), D ** -0.5, t),
            normal(g, (S, H), 0.1, t))


def rounded(ref, e, t):
    return e + half(t) * (ref.abs() + e) + 1e-38


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("S,H,D", SHAPES + TILES)
def test_forward(S, H, D, t):
    print(f"[ffn forward {S}x{H}x{D} {t}]", flush=True)
    x, wu, wg, wd, _ = make(S, H, D, t, 1)
    o, u, g, eo, eu, eg = ffn_ref(x, wu, wg, wd, t == BF)
    b = FFNBuffers(S, H, D, MD[t], device=DEV)
    b.ws.fill_(0xFF)
    check("o", b.forward(x, wu, wg, wd), o, rounded(o, eo, t))
    check("u", b.U, u, rounded(u, eu, t))
    check("g", b.G, g, rounded(g, eg, t))
    # without keeping u and g, and with an fp32 output
    f = FFNBuffers(S, H, D, MD[t], keep=False, out_f32=True, device=DEV)
    check("o fp32", f.forward(x, wu, wg, wd), o, rounded(o, eo, F32))
    assert torch.equal(f.O.to(t), b.O)


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("S,H,D", SHAPES + TILES)
def test_backward(S, H, D, t):
    print(f"[ffn backward {S}x{H}x{D} {t}]", flush=True)
    x, wu, wg, wd, do = make(S, H, D, t, 2)
    u, g = mm(x, wu).to(t), mm(x, wg).to(t)
    refs, errs = ffn_bwd_ref(do, x, wu, wg, wd, u, g, t == BF)
    b = FFNBuffers(S, H, D, MD[t], train=True, device=DEV)
    b.ws.fill_(0xFF)
    got = b.backward(do, x, wu, wg, wd, u, g)
    for n, v, r, e in zip(("dx", "dwu", "dwg", "dwd"), got, refs, errs):
        check(n, v, r, rounded(r, e, t))
    first = [v.clone() for v in got]
    got = b.backward(do, x, wu, wg, wd, u, g)
    assert all(torch.equal(p, q) for p, q in zip(first, got)), "not reproducible"
    # weight gradients as fp32: the same sums, not rounded
    f = FFNBuffers(S, H, D, MD[t], train=True, out_f32=True, device=DEV)
    got = f.backward(do, x, wu, wg, wd, u, g)
    assert got[1].dtype == F32 and torch.equal(got[0], first[0])
    assert all(torch.equal(p.to(t), q) for p, q in zip(got[1:], first[1:]))


def test_backward_parts():
    """dX alone and the weight gradients alone: the same values."""
    S, H, D = 200, 264, 392
    x, wu, wg, wd, do = make(S, H, D, BF, 3)
    u, g = mm(x, wu).to(BF), mm(x, wg).to(BF)
    b = FFNBuffers(S, H, D, train=True, device=DEV)
    want = [v.clone() for v in b.backward(do, x, wu, wg, wd, u, g)]
    for v in (b.dX, b.dW_up, b.dW_gate, b.dW_down):
        v.fill_(float("nan"))
    moe.moe_ffn_backward(b.shape, do, x, wu, wg, wd, u, g, b.dX, None, None, None, b.ws)
    assert torch.equal(b.dX, want[0]) and bool(torch.isnan(b.dW_up).all())
    b.dX.fill_(float("nan"))
    moe.moe_ffn_backward(b.shape, do, x, wu, wg, wd, u, g, None, b.dW_up, b.dW_gate, b.dW_down,
                         b.ws)
    assert bool(torch.isnan(b.dX).all())
    assert all(torch.equal(p, q) for p, q in zip((b.dW_up, b.dW_gate, b.dW_down), want[1:]))


def test_no_tokens():
    x, wu, wg, wd, _ = make(0, 64, 72, BF, 4)
    b = FFNBuffers(0, 64, 72, train=True, device=DEV)
    for v in (b.dW_up, b.dW_gate, b.dW_down):
        v.fill_(3)
    b.forward(x, wu, wg, wd)
    b.backward(x, x, wu, wg, wd)
    assert all(float(v.float().abs().max()) == 0 for v in (b.dW_up, b.dW_gate, b.dW_down))


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
def test_not_finite_values_stay_in_their_rows(t):
    """A NaN in one token reaches that token's output and dX, and no other token's;
    tiles that end inside the last rows do not spread what lies behind the arrays."""
    S, H, D = 70, 136, 200
    x, wu, wg, wd, do = make(S, H, D, t, 5)
    b = FFNBuffers(S, H, D, MD[t], train=True, device=DEV)
    o0 = b.forward(x, wu, wg, wd).clone()
    dx0 = b.backward(do, x, wu, wg, wd)[0].clone()
    x[5, 3], do[9, 0] = float("nan"), float("inf")
    keep_u, keep_g = b.U.clone(), b.G.clone()
    o = b.forward(x, wu, wg, wd)
    rows = torch.arange(S, device=DEV) != 5
    assert bool(torch.isnan(o[5]).all()) and torch.equal(o[rows], o0[rows])
    dx = b.backward(do, x, wu, wg, wd, keep_u, keep_g)[0]
    rows = torch.arange(S, device=DEV) != 9
    assert not bool(torch.isfinite(dx[9].float()).any()) and torch.equal(dx[rows], dx0[rows])


def test_saturated_activations():
    """Pre-activations far past exp's range: SiLU is 0 or the identity, its derivative 0
    or 1, with no NaN."""
    S, H, D = 4, 8, 8
    x = torch.zeros((S, H), device=DEV)
    u = torch.tensor([[-1e4, -200.0, -89.0, 0.0, 89.0, 200.0, 1e4, 3e38]] * S, device=DEV)
    g = torch.full((S, D), 2.0, device=DEV)
    eye = torch.eye(8, device=DEV)
    do = torch.ones((S, H), device=DEV)
    b = FFNBuffers(S, H, D, moe.MOE_F32, train=True, device=DEV)
    z = torch.zeros_like(eye)
    dx, _, _, dwd = b.backward(do, x, eye, z, eye, u, g)  # dX = dU
    assert torch.allclose(dx[0], torch.tensor([0., 0, 0, 1, 2, 2, 2, 2], device=DEV), atol=1e-5)
    assert bool(torch.isfinite(dx).all())


@pytest.mark.timeout(300)
def test_arrays_past_4_gib():
    """U, G and the workspace's rows exceed 4 GiB each: the last rows, and the sums over
    all rows."""
    S, H, D = (1 << 20) + 77, 8, 2056
    print(f"[ffn {S}x{H}x{D}]", flush=True)
    x, wu, wg, wd, do = make(S, H, D, BF, 6)
    b = FFNBuffers(S, H, D, train=True, out_f32=True, device=DEV)
    assert b.U.numel() * 2 > 1 << 32
    b.forward(x, wu, wg, wd)
    last = slice(S - 300, S)
    o, u, g, eo, eu, eg = ffn_ref(x[last], wu, wg, wd, True)
    check("o", b.O[last], o, rounded(o, eo, F32))
    check("u", b.U[last], u, rounded(u, eu, BF))
    got = b.backward(do, x, wu, wg, wd)
    refs, errs = ffn_bwd_ref(do[last], x[last], wu, wg, wd, b.U[last], b.G[last], True)
    check("dx", got[0][last], refs[0], rounded(refs[0], errs[0], BF))
    total, bound = 0, 0
    for i in range(0, S, 1 << 16):
        r = slice(i, min(i + (1 << 16), S))
        q, e = ffn_bwd_ref(do[r], x[r], wu, wg, wd, b.U[r], b.G[r], True)
        total = total + q[3]
        bound = bound + e[3].square()  # independent parts: their bounds add in squares
    # and the chain over all rows: at most S u of the magnitudes, here by its root (a
    # random walk of roundings), six of them
    check("dwd", got[3], total, 2 * bound.sqrt() + 6 * S ** 0.5 * 2.0 ** -24 * 30 * S ** 0.5)


def test_gradient_against_differences():
    """<gradient, v> against central differences of the library's own fp32 forward."""
    S, H, D = 24, 40, 56
    x, wu, wg, wd, c = make(S, H, D, F32, 7)
    b = FFNBuffers(S, H, D, moe.MOE_F32, train=True, device=DEV)
    b.forward(x, wu, wg, wd)
    grads = [v.clone() for v in b.backward(c, x, wu, wg, wd)]
    g = gen(8)
    for i, p in enumerate((x, wu, wg, wd)):
        v = torch.randn(p.shape, generator=g, device=DEV)
        v /= v.norm()
        e = 0.02  # fp32 forward: 1e-6 of |L| / e of noise, e^2 of third derivatives
        args = [x, wu, wg, wd]
        val = []
        for s in (e, -e):
            args[i] = p + s * v
            val.append(float((b.forward(*args).double() * c.double()).sum()))
        num = (val[0] - val[1]) / (2 * e)
        want = float((grads[i].double() * v.double()).sum())
        assert abs(num - want) < 1e-3 * max(1.0, abs(want)), (i, num, want)


def sublayer(x, gamma, beta, w, do, ln, ff):
    """A pre-norm sublayer and its gradients: y = ffn(norm(x)), then back to x."""
    y = ff.forward(ln.forward(x, gamma, beta), *w)
    grads = ff.backward(do, ln.Y, *w)
    return (y, *grads[1:], *ln.backward(grads[0], x, gamma))


def test_sublayer_together():
    """Norm and block as they are used together, forward and backward, against the same
    in 64 bits (from the kept values, so that each operator's own bound applies)."""
    from tests.ffn_util import ln_bwd_ref
    S, H, D = 150, 264, 520
    x, wu, wg, wd, do = make(S, H, D, BF, 9)
    g = gen(10)
    gamma, beta = normal(g, (H,), 0.2, BF, 1.0), normal(g, (H,), 0.2, BF)
    ln, ff = LayerNormBuffers(S, H, device=DEV), FFNBuffers(S, H, D, train=True, device=DEV)
    y, dwu, dwg, dwd, dx, dgamma, dbeta = sublayer(x, gamma, beta, (wu, wg, wd), do, ln, ff)
    o, _, _, eo, _, _ = ffn_ref(ln.Y, wu, wg, wd, True)
    check("y", y, o, rounded(o, eo, BF))
    refs, errs = ffn_bwd_ref(do, ln.Y, wu, wg, wd, ff.U, ff.G, True)
    for n, v, r, e in zip(("dy", "dwu", "dwg", "dwd"), (ff.dX, dwu, dwg, dwd), refs, errs):
        check(n, v, r, rounded(r, e, BF))
    rx, rg, rb, ex, eg, eb = ln_bwd_ref(ff.dX, x, gamma, ln.mean, ln.rstd)
    check("dx", dx, rx, rounded(rx, ex, BF))
    check("dgamma", dgamma, rg, eg)
    check("dbeta", dbeta, rb, eb)


def test_captured_sublayer_replays():
    """The whole sublayer captured in a graph, replayed with eager work of the same
    buffers' operators between the replays."""
    S, H, D = 130, 256, 392
    x, wu, wg, wd, do = make(S, H, D, BF, 11)
    g = gen(12)
    gamma, beta = normal(g, (H,), 0.2, BF, 1.0), normal(g, (H,), 0.2, BF)
    bufs = lambda: (LayerNormBuffers(S, H, device=DEV),
                    FFNBuffers(S, H, D, train=True, device=DEV))
    eager, cap = bufs(), bufs()
    args = (x, gamma, beta, (wu, wg, wd), do)
    want = [v.clone() for v in sublayer(*args, *eager)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sublayer(*args, *cap)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sublayer(*args, *cap)
    for rep in range(3):
        for v in out:
            v.fill_(float("nan"))
        cap[0].ws.fill_(0xFF)
        cap[1].ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), f"replay {rep}"
        again = sublayer(*args, *eager)
        assert all(torch.equal(p, q) for p, q in zip(again, want))


def test_two_streams_at_once():
    """Two blocks with buffers of their own on two streams."""
    S, H, D = 300, 256, 512
    sets = [make(S, H, D, BF, s) for s in (13, 14)]
    bufs = [FFNBuffers(S, H, D, train=True, device=DEV) for _ in sets]

    def step(i, stream=None):
        x, wu, wg, wd, do = sets[i]
        o = bufs[i].forward(x, wu, wg, wd, stream=stream)
        return [o, *bufs[i].backward(do, x, wu, wg, wd, stream=stream)]

    want = [[v.clone() for v in step(i)] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = [step(i, streams[i]) for i in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for a, b in zip(got, want) for p, q in zip(a, b))


def test_binding_refusals():
    x, wu, wg, wd, do = make(16, 64, 72, BF, 15)
    b = FFNBuffers(16, 64, 72, train=True, device=DEV)
    with pytest.raises(ValueError, match="W_up is"):
        b.forward(x, wu.t().contiguous(), wg, wd)
    with pytest.raises(ValueError, match="contiguous"):
        b.forward(x, torch.empty((72, 64), dtype=BF, device=DEV).t(), wg, wd)
    with pytest.raises(ValueError, match="bfloat16"):
        b.forward(x.float(), wu, wg, wd)
    with pytest.raises(ValueError, match="device memory"):
        b.forward(x.cpu(), wu, wg, wd)
    with pytest.raises(moe.MoeError, match="WORKSPACE"):
        moe.moe_ffn_forward(b.shape, x, wu, wg, wd, None, None, b.O, b.ws[:64])
    with pytest.raises(moe.MoeError, match="INVALID"):
        moe.moe_ffn_forward(b.shape, x, wu, wg, wd, b.U, None, b.O, b.ws)


# What SHAPES and TILES leave out of the plan's choices: dh, down and both weight
# gradients on the 256 x 256 tile with splits of K, down, dh and dW_down on 128 x 128 with
# splits, down on 256 x 128 with splits, up in one split over 64 rows; fp32: down and dX on
# 128 x 128 without splits, up, dh, down and dX over several row tiles of 16 with splits.
MORE_TILES = [(17, 1032, 72), (33, 136, 7176), (65, 4104, 4104), (257, 7176, 4104),
              (4100, 4104, 72), (6000, 264, 7176), (8200, 7176, 136)]


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("S,H,D", MORE_TILES)
def test_remaining_tiles(S, H, D, t):
    test_forward(S, H, D, t)
    test_backward(S, H, D, t)


@pytest.mark.timeout(300)
def test_every_weight_gradient_past_4_gib():
    """dO is zero but in 8 early rows and the 4157 whose U, G, dU, dG and h lie past 4 GiB,
    so that each weight gradient is the sum of those rows' products, within the usual
    bound of that many terms; without the rows past 4 GiB it would miss it."""
    S, H, D = (1 << 20) + 77, 8, 2056
    print(f"[ffn {S}x{H}x{D}]", flush=True)
    x, wu, wg, wd, do = make(S, H, D, BF, 16)
    past = -(-(1 << 32) // (D * 2))
    do[8:past] = 0
    live = torch.cat([torch.arange(8), torch.arange(past, S)]).to(DEV)
    assert past == 1044496 and live.numel() == 8 + S - past
    b = FFNBuffers(S, H, D, train=True, out_f32=True, device=DEV)
    b.forward(x, wu, wg, wd)
    b.ws.fill_(0xFF)
    got = b.backward(do, x, wu, wg, wd)
    refs, errs = ffn_bwd_ref(do[live], x[live], wu, wg, wd, b.U[live], b.G[live], True)
    early = ffn_bwd_ref(do[:8], x[:8], wu, wg, wd, b.U[:8], b.G[:8], True)[0]
    check("dx", got[0][live], refs[0], rounded(refs[0], errs[0], BF))
    assert not bool(got[0][8:past].any())
    for n, v, r, e, q in zip(("dwu", "dwg", "dwd"), got[1:], refs[1:], errs[1:], early[1:]):
        bound = rounded(r, e, F32)
        check(n, v, r, bound)
        assert float(((r - q).abs() > bound).double().mean()) > 0.9, n  # the bound says something


@pytest.mark.timeout(300)
def test_weights_past_4_gib():
    """Each weight and its gradient exceed 4 GiB: the first and the last 300 rows and
    columns. Small integers, and pre-activations of 32, where SiLU is the identity in fp32
    and its derivative 1, so that every sum stays an integer below 2^24 and exact."""
    S, H, D = 17, 32776, 32776
    print(f"[ffn {S}x{H}x{D}]", flush=True)
    g = gen(17)
    ints = lambda *n: torch.randint(-1, 2, n, generator=g, device=DEV, dtype=torch.int8).float()
    x, wu, wg, wd, do = ints(S, H), ints(H, D), ints(H, D), ints(D, H), ints(S, H)
    assert wu.numel() * 4 > 1 << 32
    b = FFNBuffers(S, H, D, moe.MOE_F32, train=True, device=DEV)
    b.forward(x, wu, wg, wd)
    ends = torch.cat([torch.arange(300), torch.arange(D - 300, D)]).to(DEV)
    assert torch.equal(b.U[:, ends].double(), mm(x, wu[:, ends]))
    assert torch.equal(b.G[:, ends].double(), mm(x, wg[:, ends]))
    u, gg = torch.full((S, D), 32.0, device=DEV), ints(S, D)
    dx, dwu, dwg, dwd = b.backward(do, x, wu, wg, wd, u, gg)
    dh = torch.cat([mm(do, p.t()) for p in wd.split(4096)], 1)
    du, dg = dh * gg.double(), dh * 32
    assert torch.equal(dx[:, ends].double(), mm(du, wu[ends].t()) + mm(dg, wg[ends].t()))
    xt, ht = x.t().contiguous(), (gg * 32).t().contiguous()
    for v, a, c in ((dwu, xt, du), (dwg, xt, dg), (dwd, ht, do)):
        assert torch.equal(v[ends].double(), mm(a[ends], c))
        assert torch.equal(v[:, ends].double(), mm(a, c[:, ends]))
    # the second product of the forward pass: its last columns from the kept U and G
    h = b.U.double() * torch.sigmoid(b.U.double()) * b.G.double()
    o, m = mm(h, wd[:, ends]), mm(h.abs(), wd[:, ends].abs())
    check("o", b.O[:, ends], o, (D + 8 * 600) * 2.0 ** -24 * m)  # |U| stays below 600
    assert float(b.U.abs().max()) < 600
