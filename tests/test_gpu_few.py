"""The whole MoE layer for a few tokens against 64-bit forms, and against the layer's other
entry points; with small integers exactly."""
import pytest
import torch

import sparse_expert_ffn_amd as moe
from sparse_expert_ffn_amd.layer import FewMoEBuffers, I8Weight, MoEBuffers
from tests.ffn_util import DEV, U, check, gen, half, mm, normal
from tests.test_gpu_i8 import quant_ref, weight

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
KINDS = {"bf16": BF, "f32": F32, "i8": BF}


class Layer:
    """Weights of one layer, as the entry points and the reference take them."""

    def __init__(self, g, kind, H, D, E, Ds=0):
        self.kind, self.t = kind, KINDS[kind]
        make = ((lambda K, N, n: weight(g, K, N, E=n)) if kind == "i8" else
                (lambda K, N, n: normal(g, (n, K, N), K ** -0.5, self.t)))
        self.w = [make(H, D, E), make(H, D, E), make(D, H, E)]
        self.s = [make(H, Ds, 1), make(H, Ds, 1), make(Ds, H, 1)] if Ds else []
        self.args = ([I8Weight(*v) for v in self.w + self.s] if kind == "i8" else
                     self.w + [v[0] for v in self.s])

    def ffn(self, x, m, e):
        """(y, bound before any rounding of y) of rows x through expert e of matrices m."""
        if self.kind == "i8":
            return i8_ffn(x, *((q[e], s[e]) for q, s in m))
        wu, wg, wd = (v[e] for v in m)
        H, D = wu.shape
        u, g = mm(x, wu), mm(x, wg)
        eu, eg = H * U * mm(x.abs(), wu.abs()), H * U * mm(x.abs(), wg.abs())
        a = u * torch.sigmoid(u)
        h = a * g
        eh = 1.1 * g.abs() * eu + a.abs() * eg + 8 * U * (1 + u.abs()) * h.abs()
        y = mm(h, wd)
        ey = mm(eh, wd.abs()) + D * U * mm(h.abs(), wd.abs())
        if self.kind == "bf16":  # h rounded: six standard deviations of the sum
            ey += 6 * half(BF) / 3 ** 0.5 * mm(h.square(), wd.double().square()).sqrt()
        return y, ey


def i8_ffn(x, up, gate, down):
    """As tests/test_gpu_i8.py derives it: exact integer sums, and codes of h that may move by
    one where h lies that near to a border between two."""
    q, s = quant_ref(x, 1)
    sc = s.double()
    u = mm(q, up[0]) * sc * up[1].double()
    g = mm(q, gate[0]) * sc * gate[1].double()
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
    e = sh * wd.abs().amax(0)[None] * min(moved, 6 * moved ** 0.5 + 6) + (eps + 9 * U) * o.abs() \
        + 8 * U * mm((qh * sh).abs(), wd.abs())
    return o, e


def layer_ref(ly, x, ids, wts):
    S, H = x.shape
    E = (ly.w[0][0] if ly.kind == "i8" else ly.w[0]).shape[0]
    o = torch.zeros((S, H), dtype=torch.float64, device=DEV)
    b = torch.zeros_like(o)
    for e in set(ids.flatten().tolist()):
        if not 0 <= e < E:
            continue
        s, j = (ids == e).nonzero(as_tuple=True)
        y, ey = ly.ffn(x[s].contiguous(), ly.w, e)
        w = wts[s, j].double()[:, None]
        o.index_add_(0, s, w * y)
        b.index_add_(0, s, w.abs() * (ey + 40 * U * y.abs()))
    if ly.s:
        y, ey = ly.ffn(x, ly.s, 0)
        o += y
        b += ey + 40 * U * y.abs()
    return o, b + 4 * U * o.abs() + 1e-38


def buffers(kind, S, H, D, E, k, Ds=0, **kw):
    return FewMoEBuffers(S, H, D, E, k, D_shared=Ds, i8=kind == "i8",
                         dtype=moe.MOE_F32 if kind == "f32" else moe.MOE_BF16, device=DEV, **kw)


CASES = [(1, 64, 80, 4, 2, 0), (1, 272, 144, 64, 8, 48), (5, 144, 208, 6, 3, 272),
         (40, 128, 64, 3, 2, 0), (64, 80, 144, 32, 4, 80), (3, 1024, 528, 16, 1, 16),
         (21, 208, 48, 1, 1, 0), (128, 272, 400, 8, 2, 144), (2, 2048, 768, 256, 8, 0),
         (17, 16, 16, 5, 5, 16), (7, 4112, 272, 12, 3, 0), (1, 512, 4112, 9, 2, 528),
         (128, 64, 48, 40, 32, 32)]


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("S,H,D,E,k,Ds", CASES)
def test_given_routing(S, H, D, E, k, Ds, kind):
    """With a padded token, slots without an expert, weights that are not finite there."""
    print(f"[few S={S} H={H} D={D} E={E} k={k} Ds={Ds} {kind}]", flush=True)
    g = gen(1)
    ly = Layer(g, kind, H, D, E, Ds)
    x = normal(g, (S, H), 1.0, ly.t)
    ids = torch.argsort(torch.rand((S, E), generator=g, device=DEV), 1)[:, :k].int().contiguous()
    wts = torch.rand((S, k), generator=g, device=DEV)
    if S > 2:
        ids[1] = -1
        ids[2, 0] = E + 3
        wts[2, 0] = float("nan")
    for out_f32 in ([True, False] if kind != "f32" else [False]):
        b = buffers(kind, S, H, D, E, k, Ds, out_f32=out_f32)
        b.ws.fill_(0xFF)
        o = b.forward(x, *ly.args, topk_ids=ids, topk_weights=wts)
        ref, e = layer_ref(ly, x, ids, wts)
        check("o", o, ref, e + half(o.dtype) * (ref.abs() + e))
        if S > 2 and not Ds:
            assert not bool(o[1].any())
        again = buffers(kind, S, H, D, E, k, Ds, out_f32=out_f32)
        again.ws.fill_(0x01)
        assert torch.equal(again.forward(x, *ly.args, topk_ids=ids, topk_weights=wts), o)


def route_ref(x, wr, bias, k, renormalize):
    """Scores in 64 bits, rounded to fp32 before the fp32 bias is added."""
    s = mm(x, wr).float()
    if bias is not None:
        s = s + bias
    top, ids = (v[:, :k] for v in torch.sort(s, dim=1, descending=True, stable=True))
    e = torch.exp(top.double() - top[:, :1].double())
    den = e.sum(1) if renormalize else torch.exp(s.double() - top[:, :1].double()).sum(1)
    return s, ids.int(), e / den[:, None]


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("S,H,E,k,bias,renorm", [
    (1, 2048, 256, 8, False, 1), (3, 272, 6, 2, True, 1), (64, 2048, 256, 8, True, 0),
    (33, 528, 25, 4, True, 1), (128, 144, 1024, 32, False, 1), (5, 7168, 100, 3, False, 0),
    (2, 16, 1, 1, True, 1), (19, 256, 129, 5, True, 1)])
def test_router(S, H, E, k, bias, renorm, kind):
    """Ids: those of the 64-bit scores, but where two scores are nearer than the sum's error;
    weights to the scores' error; the output follows the routing that was written."""
    print(f"[router S={S} H={H} E={E} k={k} {kind}]", flush=True)
    g = gen(2)
    D = 32
    ly = Layer(g, kind, H, D, E)
    x = normal(g, (S, H), 1.0, ly.t)
    wr = normal(g, (H, E), H ** -0.5, ly.t)
    bs = torch.randn(E, generator=g, device=DEV) if bias else None
    b = buffers(kind, S, H, D, E, k, renormalize=renorm)
    b.ws.fill_(0xFF)
    o = b.run(x, wr, *ly.args, router_bias=bs)
    s, ids, w = route_ref(x, wr, bs, k, renorm)
    # a score: up to 256 terms in fp32, the sums in 64 bits, two roundings
    es = 258 * U * mm(x.abs(), wr.abs()) + 2 * U * s.abs().double()
    got = torch.gather(s, 1, b.topk_ids.long()).double()
    want = torch.gather(s, 1, ids.long()).double()
    assert bool(((got - want).abs() <= 2 * es.amax(1, keepdim=True)).all())
    assert all(len(set(r)) == k for r in b.topk_ids.tolist())
    assert int((b.topk_ids != ids).sum()) <= 2
    # exp of differences of two scores, over sums of such
    check("w", b.topk_weights, torch.where(b.topk_ids == ids, w, b.topk_weights.double()),
          (4 * es.amax(1, keepdim=True) + 4 * U) * w + 1e-38)
    ref, e = layer_ref(ly, x, b.topk_ids, b.topk_weights)
    check("o", o, ref, e + half(o.dtype) * (ref.abs() + e))


def test_router_ties_and_nan():
    """Equal scores: the lower index; a NaN score ranks last; a NaN token stays alone."""
    g = gen(3)
    S, H, D, E, k = 4, 64, 32, 40, 3
    ly = Layer(g, "bf16", H, D, E)
    x = torch.ones((S, H), dtype=BF, device=DEV)
    wr = torch.zeros((H, E), dtype=BF, device=DEV)
    wr[:, 30], wr[:, 7], wr[:, 20], wr[:, 21] = 1.0, 1.0, 0.5, 0.5
    b = buffers("bf16", S, H, D, E, k)
    b.run(x, wr, *ly.args)
    assert b.topk_ids.tolist() == [[7, 30, 20]] * S
    bias = torch.zeros(E, device=DEV)
    bias[7] = float("nan")
    o = b.run(x, wr, *ly.args, router_bias=bias).clone()
    assert b.topk_ids.tolist() == [[30, 20, 21]] * S
    x[2, 5] = float("nan")
    o2 = b.run(x, wr, *ly.args, router_bias=bias)
    keep = torch.tensor([0, 1, 3], device=DEV)
    assert torch.equal(o[keep], o2[keep]) and bool(torch.isnan(o2[2]).all())


@pytest.mark.parametrize("kind", list(KINDS))
def test_tokens_do_not_meet(kind):
    """A token of infinities or NaN in the rows of an expert leaves the others' as they were."""
    g = gen(4)
    S, H, D, E, k = 12, 144, 80, 4, 2
    ly = Layer(g, kind, H, D, E, 48)
    x = normal(g, (S, H), 1.0, ly.t)
    ids = torch.randint(0, E, (S, k), generator=g, device=DEV, dtype=torch.int32)
    wts = torch.rand((S, k), generator=g, device=DEV)
    b = buffers(kind, S, H, D, E, k, 48)
    o = b.forward(x, *ly.args, topk_ids=ids, topk_weights=wts).clone()
    x[3, 7], x[9, H - 1] = float("nan"), float("inf")
    o2 = b.forward(x, *ly.args, topk_ids=ids, topk_weights=wts)
    keep = torch.ones(S, dtype=torch.bool, device=DEV)
    keep[3] = keep[9] = False
    assert torch.equal(o[keep], o2[keep]) and bool(torch.isnan(o2[3]).all())
    assert not bool(torch.isfinite(o2[9]).any())


def test_exact_integers():
    """Small integers in fp32 with G = 1 and U large (SiLU(U) = U to fp32): every sum is
    exact."""
    g = gen(5)
    S, H, D, E, k = 23, 136, 200, 6, 2
    x = torch.zeros((S, H), device=DEV)
    x[:, 0] = torch.randint(30, 40, (S,), generator=g, device=DEV).float()
    x[:, 1] = 1.0
    wu, wg = torch.zeros((E, H, D), device=DEV), torch.zeros((E, H, D), device=DEV)
    wu[:, 0] = 1.0  # u = 30 .. 39
    wg[:, 1] = torch.randint(-2, 3, (E, D), generator=g, device=DEV).float()
    wd = torch.randint(-3, 4, (E, D, H), generator=g, device=DEV).float()
    ids = torch.randint(0, E, (S, k), generator=g, device=DEV, dtype=torch.int32)
    wts = torch.randint(-2, 3, (S, k), generator=g, device=DEV).float()
    b = buffers("f32", S, H, D, E, k)
    o = b.forward(x, wu, wg, wd, topk_ids=ids, topk_weights=wts)
    ref = torch.zeros((S, H), dtype=torch.float64, device=DEV)
    for t in range(S):
        for j in range(k):
            e = int(ids[t, j])
            h = x[t, 0].double() * wg[e, 1].double()
            ref[t] += wts[t, j].double() * (h @ wd[e].double())
    # SiLU(u) = u / (1 + exp(-u)), exp(-30) < 2^-43: u (rcp(1) = 1)
    assert torch.equal(o.double(), ref)


def test_same_expert_twice_and_all_on_one():
    g = gen(6)
    S, H, D, E, k = 37, 64, 80, 4, 3
    for kind in KINDS:
        ly = Layer(g, kind, H, D, E)
        x = normal(g, (S, H), 1.0, ly.t)
        ids = torch.full((S, k), 2, dtype=torch.int32, device=DEV)
        ids[:, 2] = 0
        wts = torch.rand((S, k), generator=g, device=DEV)
        b = buffers(kind, S, H, D, E, k)
        o = b.forward(x, *ly.args, topk_ids=ids, topk_weights=wts)
        ref, e = layer_ref(ly, x, ids, wts)
        check(kind, o, ref, e + half(o.dtype) * (ref.abs() + e))


def test_no_expert_at_all():
    ly = Layer(gen(7), "bf16", 64, 32, 4)
    b = buffers("bf16", 3, 64, 32, 4, 2)
    o = b.forward(torch.ones((3, 64), dtype=BF, device=DEV), *ly.args,
                  topk_ids=torch.full((3, 2), -1, dtype=torch.int32, device=DEV),
                  topk_weights=torch.full((3, 2), float("inf"), device=DEV))
    assert not bool(o.any())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_agrees_with_the_layer(kind):
    """MoEBuffers on the same inputs: the same routing, outputs to two roundings."""
    g = gen(8)
    S, H, D, E, k, Ds = 24, 256, 128, 16, 4, 64
    ly = Layer(g, kind, H, D, E, Ds)
    x, wr = normal(g, (S, H), 1.0, ly.t), normal(g, (H, E), 0.1, ly.t)
    b = buffers(kind, S, H, D, E, k, Ds, out_f32=True)
    m = MoEBuffers(S, H, D, E, k, D_shared=Ds, block_size=16, out_f32=True, device=DEV,
                   dtype=moe.MOE_F32 if kind == "f32" else moe.MOE_BF16)
    o, r = b.run(x, wr, *ly.args), m.run(x, wr, *ly.args)
    assert torch.equal(b.topk_ids, m.topk_ids)
    _, e = layer_ref(ly, x, b.topk_ids, b.topk_weights)
    check("o", o, r.double(), 2 * e + 8 * U * r.double().abs())


@pytest.mark.parametrize("kind", list(KINDS))
def test_captured(kind):
    """Two layers in one graph (the second's input the first's output), replayed with other
    inputs and with eager work in between."""
    g = gen(9)
    S, H, D, E, k = 6, 256, 128, 16, 4
    ly, l2 = Layer(g, kind, H, D, E, 48), Layer(g, kind, H, D, E)
    x, wr = normal(g, (S, H), 1.0, ly.t), normal(g, (H, E), 0.1, ly.t)
    mk = lambda: (buffers(kind, S, H, D, E, k, 48), buffers(kind, S, H, D, E, k))
    step = lambda a, b: b.run(a.run(x, wr, *ly.args), wr, *l2.args)
    cap, eager = mk(), mk()
    step(*cap)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*cap)
    x0 = x.clone()
    for rep in range(4):
        x.copy_(x0.roll(rep, 0) * (rep + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cap[1].O, step(*eager)), rep


def test_two_streams_at_once():
    """Calls that run at the same time, each with buffers of its own."""
    g = gen(10)
    S, H, D, E, k = 9, 1024, 512, 32, 4
    ly = Layer(g, "bf16", H, D, E)
    xs = [normal(g, (S, H), 1.0, BF) for _ in range(4)]
    wr = normal(g, (H, E), 0.05, BF)
    bs = [buffers("bf16", S, H, D, E, k) for _ in range(4)]
    want = [bs[0].run(x, wr, *ly.args).clone() for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for rep in range(5):
        for x, b, st in zip(xs, bs, streams):
            b.run(x, wr, *ly.args, stream=st)
    torch.cuda.synchronize()
    for b, w in zip(bs, want):
        assert torch.equal(b.O, w)


def test_no_tokens():
    ly = Layer(gen(11), "bf16", 64, 32, 4)
    e = lambda *n, t=BF: torch.empty(n, dtype=t, device=DEV)
    moe.moe_few_forward(moe.make_shape(0, 64, 32, 4, 2), e(0, 64), e(64, 4), None, *ly.args, None,
                        None, None, e(0, 2, t=torch.int32), e(0, 2, t=F32), e(0, 64),
                        e(256, t=torch.uint8))


def test_binding_refusals():
    g = gen(12)
    ly, l8 = Layer(g, "bf16", 64, 32, 4, 16), Layer(g, "i8", 64, 32, 4, 16)
    x = torch.zeros((2, 64), dtype=BF, device=DEV)
    wr = torch.zeros((64, 4), dtype=BF, device=DEV)
    b, c = buffers("bf16", 2, 64, 32, 4, 2, 16), buffers("i8", 2, 64, 32, 4, 2, 16)
    with pytest.raises(TypeError, match="W_up must be a tensor"):
        b.run(x, wr, *l8.args)
    with pytest.raises(TypeError, match="I8Weight"):
        c.run(x, wr, *ly.args)
    with pytest.raises(ValueError, match="W_router"):
        b.run(x, wr[:, :3].contiguous(), *ly.args)
    with pytest.raises(ValueError, match="contiguous"):
        b.run(x, wr.t().contiguous().t(), *ly.args)
    with pytest.raises(moe.MoeError, match="INVALID"):
        b.run(x, wr, *ly.args[:3])
    with pytest.raises(ValueError, match="topk_ids"):
        b.forward(x, *ly.args, topk_ids=b.topk_ids.long())
    with pytest.raises(ValueError, match="A is"):
        b.run(x.float(), wr, *ly.args)
    with pytest.raises(ValueError, match="W_down"):
        c.run(x, wr, *l8.args[:2], l8.args[0], *l8.args[3:])
    with pytest.raises(TypeError, match="required"):
        b.run(x, wr, None, *ly.args[1:])
