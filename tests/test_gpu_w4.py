"""4-bit weights: quantisation, packing, the product for few rows and the MoE
layer's experts, against 64-bit forms; where every sum is a small integer, exactly."""
import pytest
import torch

import sparse_expert_ffn_amd as moe
from sparse_expert_ffn_amd.layer import W4MoEBuffers, W4Weight
from tests.ffn_util import DEV, U, check, dequant, gen, half, mm, normal, w4, w4_bound

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("E,K,N,group", [(1, 8, 8, 32), (2, 200, 24, 64), (3, 256, 136, 128),
                                         (1, 1032, 40, 32)])
def test_quantize(E, K, N, group, t):
    g = gen(1)
    w = normal(g, (E, K, N), 0.3, t)
    w[0, :group, 0] = 0  # an all-zero group
    w[0, 0, 1] = -5      # a large negative value
    codes = torch.empty((E, K, N), dtype=torch.uint8, device=DEV)
    scales = torch.empty((E, -(-K // group), N), dtype=BF, device=DEV)
    moe.moe_quantize_w4(w, group, codes, scales)
    for q in range(scales.shape[1]):
        part = w[:, q * group:(q + 1) * group].float()
        s = (part.abs().amax(1) / 7).to(BF)
        assert torch.equal(scales[:, q], s)
        s = s.float()[:, None]
        want = torch.where(s > 0, torch.round(part / s), 0.0).clamp(-8, 7) + 8
        assert torch.equal(codes[:, q * group:(q + 1) * group].float(), want)
    # and back: off by half a step (the scale's rounding can clamp 2^-8 of the largest)
    back = dequant(codes, scales, group)
    s = scales.double().repeat_interleave(group, dim=1)[:, :K]
    assert bool(((back - w.double()).abs() <= s * (0.5 + 7 * 2.0 ** -8 + 1e-6)).all())


@pytest.mark.parametrize("E,K,N,group", [(1, 128, 16, 128), (2, 136, 24, 32), (1, 264, 40, 64)])
def test_packed_layout(E, K, N, group):
    """Byte by byte as the header describes it."""
    codes, scales = w4(gen(2), E, K, N, group)
    p = W4Weight(codes, scales, group).packed.cpu()
    c, s = codes.cpu(), scales.cpu().view(torch.int16)
    nt, kt, tb = -(-N // 16), -(-K // 128), 1024 + 128 // group * 32
    assert p.numel() == E * nt * kt * tb
    for e in range(E):
        for ct in range(nt):
            for k in range(kt):
                at = ((e * nt + ct) * kt + k) * tb
                words = p[at:at + 1024].view(torch.int32).view(64, 4)
                sc = p[at + 1024:at + tb].view(torch.int16).view(16, -1)
                for lane in range(0, 64, 5):
                    n, q = ct * 16 + lane % 16, lane // 16
                    for i in range(4):
                        v = 0
                        for j in range(8):
                            r = k * 128 + 32 * i + 8 * q + j
                            code = int(c[e, r, n]) if r < K and n < N else 8
                            v |= code << (4 * (j // 2) + 16 * (j % 2))
                        v = ((v << 3) | (v >> 29)) & 0xFFFFFFFF
                        assert int(words[lane, i]) & 0xFFFFFFFF == v
                    for gi in range(sc.shape[1]):
                        gg = k * (128 // group) + gi
                        want = int(s[e, gg, n]) if gg < s.shape[1] and n < N else 0
                        assert int(sc[lane % 16, gi]) == want


SIZES = [(1, 8, 8), (1, 128, 16), (1, 2048, 1000), (2, 136, 24), (3, 2056, 264), (15, 200, 72),
         (16, 1024, 128), (17, 264, 40), (33, 520, 136), (70, 72, 200), (1, 7168, 64)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("S,K,N", SIZES)
def test_matvec(S, K, N, group):
    print(f"[matvec {S}x{K}x{N} group {group}]", flush=True)
    g = gen(3)
    codes, scales = w4(g, 1, K, N, group)
    x = normal(g, (S, K), 1.0, BF)
    w = W4Weight(codes, scales, group)
    ref = mm(x, dequant(codes, scales, group)[0])
    e = w4_bound(x, codes[0], scales[0], group)
    for t in (BF, F32):
        y = torch.full((S, N), float("nan"), dtype=t, device=DEV)
        moe.moe_w4_matvec(x, w, y)
        check(str(t), y, ref, e + half(t) * (ref.abs() + e) + 1e-38)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_matvec_exact_integers(group):
    """Integer rows and scales of 2^-3: every partial sum is exact, so is the result.
    K leaves a short last group and a short last tile."""
    g = gen(4)
    S, K, N = 21, 1000, 88
    codes = torch.randint(0, 256, (1, K, N), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.full((1, -(-K // group), N), 0.125, dtype=BF, device=DEV)
    x = torch.randint(-9, 10, (S, K), generator=g, device=DEV).to(BF)
    y = torch.empty((S, N), device=DEV)
    moe.moe_w4_matvec(x, W4Weight(codes, scales, group), y)
    assert torch.equal(y.double(), mm(x, dequant(codes & 15, scales, group)[0]))


@pytest.mark.parametrize("S,E", [(1, 4), (9, 64), (40, 3), (64, 5), (33, 1), (5, 5)])
def test_matvec_by_expert(S, E):
    """Rows with a matrix each: shared ones (more than 16 rows of one), the same one
    twice, and ids outside [0, E), whose rows are zeros."""
    g = gen(5)
    K, N, group = 264, 72, 64
    codes, scales = w4(g, E, K, N, group)
    x = normal(g, (S, K), 1.0, BF)
    ids = torch.randint(0, E, (S,), generator=g, device=DEV, dtype=torch.int32)
    ids[S // 2:S // 2 + 3] = torch.tensor([-1, E, 0x7FFFFFFF], device=DEV)[:S - S // 2]
    if S > 30:
        ids[:20] = E - 1
    y = torch.full((S, N), float("nan"), device=DEV)
    moe.moe_w4_matvec(x, W4Weight(codes, scales, group), y, expert_ids=ids)
    for s, e in enumerate(ids.tolist()):
        if not 0 <= e < E:
            assert torch.equal(y[s], torch.zeros(N, device=DEV)), s
            continue
        ref = mm(x[s:s + 1], dequant(codes, scales, group)[e])
        b = w4_bound(x[s:s + 1], codes[e], scales[e], group)
        check(f"row {s}", y[s:s + 1], ref, b + half(F32) * ref.abs())


def test_matvec_rows_do_not_meet():
    """A NaN row stays alone among the rows of its block; the same row gives the same
    bits wherever it stands."""
    g = gen(6)
    codes, scales = w4(g, 1, 512, 64, 32)
    w = W4Weight(codes, scales, 32)
    x = normal(g, (16, 512), 1.0, BF)
    y, z, one = (torch.empty((n, 64), device=DEV) for n in (16, 16, 1))
    moe.moe_w4_matvec(x, w, y)
    x2 = x.flip(0).contiguous()
    x2[3, 100] = float("nan")
    moe.moe_w4_matvec(x2, w, z)
    keep = torch.arange(16, device=DEV) != 3
    assert torch.equal(z[keep], y.flip(0)[keep]) and bool(torch.isnan(z[3]).all())
    moe.moe_w4_matvec(x[5:6], w, one)
    assert torch.equal(one[0], y[5])


def layer_ref(x, up, gate, down, sh, ids, wts, group):
    """(o, bound before rounding)."""
    S, H = x.shape
    o = torch.zeros((S, H), dtype=torch.float64, device=DEV)
    b = torch.zeros_like(o)
    q = 6 * half(BF) / 3 ** 0.5

    def ffn(xr, u_, g_, d_, e):
        (cu, su), (cg, sg), (cd, sd) = u_, g_, d_
        wd = dequant(cd, sd, group)[e]
        u, g = mm(xr, dequant(cu, su, group)[e]), mm(xr, dequant(cg, sg, group)[e])
        eu = w4_bound(xr, cu[e], su[e], group)
        eg = w4_bound(xr, cg[e], sg[e], group)
        a = u * torch.sigmoid(u)
        h = a * g
        eh = 1.1 * g.abs() * eu + a.abs() * eg + 8 * U * (1 + u.abs()) * h.abs()
        y = mm(h, wd)
        ey = mm(eh, wd.abs()) + w4_bound(h, cd[e], sd[e], group) \
            + q * mm(h.square(), wd.square()).sqrt()
        return y, ey

    for s in range(S):
        for j, e in enumerate(ids[s].tolist()):
            if not 0 <= e < up[0].shape[0]:
                continue
            y, ey = ffn(x[s:s + 1], up, gate, down, e)
            w = float(wts[s, j])
            o[s] += w * y[0]
            b[s] += abs(w) * (ey[0] + 40 * U * y[0].abs())
    if sh is not None:
        y, ey = ffn(x, *sh, 0)
        o += y
        b += ey + 40 * U * y.abs()
    return o, b + 4 * U * o.abs()


CASES = [(1, 64, 72, 4, 2, 0, 32), (1, 264, 136, 64, 8, 40, 64), (5, 136, 200, 6, 3, 264, 128),
         (40, 128, 64, 3, 2, 0, 64), (64, 72, 136, 32, 4, 72, 32), (3, 1024, 520, 16, 1, 8, 128),
         (21, 200, 40, 1, 1, 0, 128)]


@pytest.mark.parametrize("S,H,D,E,k,Ds,group", CASES)
def test_layer(S, H, D, E, k, Ds, group):
    print(f"[w4 layer S={S} H={H} D={D} E={E} k={k} Ds={Ds} group {group}]", flush=True)
    g = gen(7)
    up, gate, down = w4(g, E, H, D, group), w4(g, E, H, D, group), w4(g, E, D, H, group)
    sh = (w4(g, 1, H, Ds, group), w4(g, 1, H, Ds, group), w4(g, 1, Ds, H, group)) if Ds else None
    x = normal(g, (S, H), 1.0, BF)
    b = W4MoEBuffers(S, H, D, E, k, D_shared=Ds, group=group, out_f32=True, device=DEV)
    b.route(logits_in=torch.randn((S, E), generator=g, device=DEV))
    if S > 2:  # a padded token, a slot without an expert whose weight is not finite
        b.topk_ids[1] = -1
        b.topk_ids[2, 0] = E + 3
        b.topk_weights[2, 0] = float("nan")
    packed = [W4Weight(*p, group=group) for p in (up, gate, down)]
    spacked = [W4Weight(*p, group=group) for p in sh] if Ds else []
    b.ws.fill_(0xFF)
    o = b.forward(x, *packed, *spacked)
    ref, e = layer_ref(x, up, gate, down, sh, b.topk_ids, b.topk_weights, group)
    check("o", o, ref, e + half(F32) * ref.abs())
    if S > 2 and not Ds:
        assert torch.equal(o[1], torch.zeros(H, device=DEV))
    f = W4MoEBuffers(S, H, D, E, k, D_shared=Ds, group=group, device=DEV)
    f.forward(x, *packed, *spacked, topk_ids=b.topk_ids, topk_weights=b.topk_weights)
    assert torch.equal(f.O, o.to(BF))


def test_layer_same_expert_twice_and_all_on_one():
    """Ids a router does not give but the call allows: an expert twice in one token, and
    every token on one expert (more than 16 rows)."""
    g = gen(8)
    S, H, D, E, k, group = 37, 64, 72, 4, 3, 32
    up, gate, down = w4(g, E, H, D, group), w4(g, E, H, D, group), w4(g, E, D, H, group)
    x = normal(g, (S, H), 1.0, BF)
    ids = torch.full((S, k), 2, dtype=torch.int32, device=DEV)
    ids[:, 2] = 0
    wts = torch.rand((S, k), generator=g, device=DEV)
    b = W4MoEBuffers(S, H, D, E, k, group=group, out_f32=True, device=DEV)
    o = b.forward(x, *(W4Weight(*p, group=group) for p in (up, gate, down)), topk_ids=ids,
                  topk_weights=wts)
    ref, e = layer_ref(x, up, gate, down, None, ids, wts, group)
    check("o", o, ref, e + half(F32) * ref.abs())


def test_layer_run_captured():
    """Router and experts as one step (quantised from bf16 weights), eager and as a graph
    replayed with other routings in between."""
    g = gen(9)
    S, H, D, E, k, group = 6, 256, 128, 16, 4, 64
    make = lambda K, N: W4Weight.quantize(normal(g, (E, K, N), K ** -0.5, BF), group)
    w = (make(H, D), make(H, D), make(D, H))
    x, wr = normal(g, (S, H), 1.0, BF), normal(g, (H, E), 0.1, BF)
    b, c = (W4MoEBuffers(S, H, D, E, k, group=group, device=DEV) for _ in range(2))
    want = b.run(x, wr, *w).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(x, wr, *w)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(x, wr, *w)
    x0 = x.clone()
    for rep in range(3):
        x.copy_(x0 * (rep + 1) if rep < 2 else x0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.O, b.run(x, wr, *w)), rep
    assert torch.equal(c.O, want)


def test_no_rows():
    codes, scales = w4(gen(10), 1, 64, 16, 32)
    w = W4Weight(codes, scales, 32)
    moe.moe_w4_matvec(torch.empty((0, 64), dtype=BF, device=DEV), w,
                      torch.empty((0, 16), dtype=BF, device=DEV))


def test_binding_refusals():
    codes, scales = w4(gen(11), 2, 64, 16, 32)
    w = W4Weight(codes, scales, 32)
    x, y = torch.zeros((2, 64), dtype=BF, device=DEV), torch.zeros((2, 16), dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="columns"):
        moe.moe_w4_matvec(x[:, :32].contiguous(), w, y)
    with pytest.raises(ValueError, match="expert_ids"):
        moe.moe_w4_matvec(x, w, y, expert_ids=torch.zeros(2, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError, match="scales"):
        W4Weight(codes, scales[:, :1], 32)
    with pytest.raises(moe.MoeError, match="INVALID"):
        W4Weight(codes, torch.zeros((2, 4, 16), dtype=BF, device=DEV), 16)
    b = W4MoEBuffers(2, 64, 16, 2, 1, group=32, device=DEV)
    with pytest.raises(ValueError, match="W_down"):
        b.forward(x, w, w, w)


@pytest.mark.parametrize("as_int", [False, True], ids=["stream", "handle"])
def test_quantize_on_another_stream(as_int):
    """What quantize allocates on the way is not reused while that stream's work runs."""
    W = normal(gen(12), (4, 512, 256), 0.05, BF)
    want = W4Weight.quantize(W, 64).packed.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # work ahead of it: some milliseconds
        a = torch.ones((4096, 4096), device=DEV)
        for _ in range(20):
            a = a @ a * 0.0
    w = W4Weight.quantize(W, 64, stream=side.cuda_stream if as_int else side)
    junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
            for n in (W.numel(), W.numel() // 32) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(w.packed, want) and len(junk) == 8


def test_layer_many_slots():
    """More slots to a token than the combine loads at a time, few tokens and many."""
    g = gen(13)
    H, D, E, k, group = 64, 40, 24, 19, 32
    up, gate, down = w4(g, E, H, D, group), w4(g, E, H, D, group), w4(g, E, D, H, group)
    packed = [W4Weight(*p, group=group) for p in (up, gate, down)]
    for S in (1, 30):
        x = normal(g, (S, H), 1.0, BF)
        b = W4MoEBuffers(S, H, D, E, k, group=group, out_f32=True, device=DEV)
        b.route(logits_in=torch.randn((S, E), generator=g, device=DEV))
        b.topk_ids[0, 8] = -1
        o = b.forward(x, *packed)
        ref, e = layer_ref(x, up, gate, down, None, b.topk_ids, b.topk_weights, group)
        check("o", o, ref, e + half(F32) * ref.abs())


def _busy(n=20):
    """Some milliseconds of work on the current stream; its result is 0."""
    a = torch.ones((4096, 4096), device=DEV)
    for _ in range(n):
        a = a @ a * 0.0
    return a[0, 0]


@pytest.mark.parametrize("as_int", [False, True], ids=["stream", "handle"])
def test_pack_on_another_stream(as_int):
    """The packed weight takes no block that the current stream's work still writes, and
    codes and scales may be released while the other stream's work reads them."""
    codes, scales = w4(gen(14), 4, 512, 256, 64)
    want = W4Weight(codes, scales, 64).packed.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    zero = _busy()
    freed = torch.empty_like(want)
    freed.copy_((zero + 255).expand(freed.shape))  # behind the work
    del freed
    w = W4Weight(codes, scales, 64, stream=side.cuda_stream if as_int else side)
    torch.cuda.synchronize()
    assert torch.equal(w.packed, want)
    with torch.cuda.stream(side):
        _busy()
    w = W4Weight(codes, scales, 64, stream=side.cuda_stream if as_int else side)
    sizes = (codes.numel(), scales.numel() * 2)
    del codes, scales
    junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(w.packed, want) and len(junk) == 8


def test_released_weight_is_not_overwritten_while_it_is_read():
    """A weight made on another stream, dropped with a product of the current stream still
    to read it: the next weight made there does not take its place before."""
    g = gen(15)
    first, second = w4(g, 2, 512, 256, 64), w4(g, 2, 512, 256, 64)
    x = normal(g, (5, 512), 1.0, BF)
    want, y = torch.empty((5, 256), device=DEV), torch.empty((5, 256), device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    w = W4Weight(*first, 64, stream=side)
    torch.cuda.synchronize()
    moe.moe_w4_matvec(x, w, want)
    torch.cuda.synchronize()
    _busy()
    moe.moe_w4_matvec(x, w, y)
    del w
    w = W4Weight(*second, 64, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    moe.moe_w4_matvec(x, w, y)
    assert not torch.equal(y, want)
