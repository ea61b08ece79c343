"""The decode operators together, as a serving step calls them, and operands of more than
4 GiB."""
import pytest
import torch

import sparse_expert_ffn_amd as moe
from sparse_expert_ffn_amd.layer import (FewMoEBuffers, I8FFNBuffers, I8LinearBuffers, I8Weight,
                                         LayerNormBuffers)
from tests.ffn_util import DEV, check, gen, half, normal
from tests.test_gpu_few import Layer, layer_ref
from tests.test_gpu_i8 import ffn_ref, product, quant_ref, weight

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Block:
    """norm -> 8-bit product -> norm -> MoE layer (8-bit experts) -> 8-bit gated block."""

    def __init__(self, S, H, D, E, k, Ds):
        b = dict(device=DEV)
        self.n1, self.n2 = LayerNormBuffers(S, H, **b), LayerNormBuffers(S, H, **b)
        self.lin = I8LinearBuffers(S, H, H, **b)
        self.moe = FewMoEBuffers(S, H, D, E, k, D_shared=Ds, i8=True, **b)
        self.ffn = I8FFNBuffers(S, H, D, out_f32=True, **b)

    def run(self, x, p):
        y = self.lin.run(self.n1.forward(x, *p.norm), p.lin)
        y = self.moe.run(self.n2.forward(y, *p.norm), p.router, *p.experts.args)
        return self.ffn.forward(y, *p.ffn)


class Params:
    def __init__(self, g, H, D, E, Ds):
        self.norm = [(1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(BF),
                     (0.1 * torch.randn(H, generator=g, device=DEV)).to(BF)]
        self.raw_lin = weight(g, H, H)
        self.raw_ffn = [weight(g, H, D), weight(g, H, D), weight(g, D, H)]
        self.lin = I8Weight(*self.raw_lin)
        self.ffn = [I8Weight(*w) for w in self.raw_ffn]
        self.experts = Layer(g, "i8", H, D, E, Ds)
        self.router = normal(g, (H, E), H ** -0.5, BF)


@pytest.mark.parametrize("S,H,D,E,k,Ds", [(1, 512, 272, 32, 4, 144), (13, 272, 144, 12, 3, 48),
                                          (64, 528, 208, 40, 8, 0), (100, 144, 400, 6, 3, 80)])
def test_block(S, H, D, E, k, Ds):
    """Each operator on what the one before it wrote, against the 64-bit forms; the whole in a
    graph, replayed on other inputs, as eager calls."""
    print(f"[block S={S} H={H} D={D} E={E} k={k} Ds={Ds}]", flush=True)
    g = gen(20)
    p = Params(g, H, D, E, Ds)
    x = normal(g, (S, H), 1.0, BF)
    b = Block(S, H, D, E, k, Ds)
    o = b.run(x, p)
    q, s = quant_ref(b.n1.Y, 1)
    ref, e = product(q, s[:, 0], p.raw_lin)
    check("product", b.lin.Y, ref, e + half(BF) * (ref.abs() + e))
    ref, e = layer_ref(p.experts, b.n2.Y, b.moe.topk_ids, b.moe.topk_weights)
    check("layer", b.moe.O, ref, e + half(BF) * (ref.abs() + e))
    ref, e = ffn_ref(b.moe.O, *p.raw_ffn)
    check("block", o, ref, e + half(F32) * (ref.abs() + e))

    cap = Block(S, H, D, E, k, Ds)
    cap.run(x, p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap.run(x, p)
    x0 = x.clone()
    for rep in range(4):
        x.copy_(x0.roll(rep, 1) * (1 + rep))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cap.ffn.O, b.run(x, p)), rep


def test_rows_beyond_4_gib():
    """Rows whose values and codes lie behind 2^32 bytes: as the same rows alone."""
    S, K, N = 530001, 8192, 24
    print(f"[rows {S}x{K}]", flush=True)
    g = gen(21)
    x = torch.empty((S, K), dtype=BF, device=DEV).normal_(generator=g)
    codes = torch.empty((S, K), dtype=torch.int8, device=DEV)
    scales = torch.empty(S, device=DEV)
    moe.moe_quantize_i8_rows(x, codes, scales)
    at = torch.tensor([0, 1, 262143, 262144, 262145, 524287, 524288, 524289, S - 1], device=DEV)
    q, s = quant_ref(x[at], 1)
    assert torch.equal(codes[at], q) and torch.equal(scales[at], s[:, 0])
    w = I8Weight(*weight(g, K, N))
    alone = I8LinearBuffers(len(at), K, N, device=DEV).run(x[at], w)
    for xx, ss in ((x, None), (codes, scales)):
        b = I8LinearBuffers(S, K, N, device=DEV)
        assert torch.equal(b.run(xx, w, ss)[at], alone)


def test_experts_beyond_4_gib():
    """The last of the experts whose weights take more than 2^32 bytes: as that one alone."""
    E, H, D = 36, 8192, 16384
    print(f"[experts {E}x{H}x{D}]", flush=True)
    g = gen(22)
    W = [torch.empty((E, *n), dtype=BF, device=DEV).normal_(generator=g).mul_(n[0] ** -0.5)
         for n in ((H, D), (H, D), (D, H))]
    x = normal(g, (2, H), 1.0, BF)
    wts = torch.tensor([[0.7], [0.4]], device=DEV)
    last = torch.full((2, 1), E - 1, dtype=torch.int32, device=DEV)
    first = torch.zeros_like(last)
    one = [w[-1:].clone() for w in W]
    for i8 in (False, True):
        many = [I8Weight.quantize(w) for w in W] if i8 else W
        few = [I8Weight.quantize(w) for w in one] if i8 else one
        if i8:
            for a, b in zip(many, few):
                assert torch.equal(a.packed[-b.nbytes:], b.packed)
        for S in (1, 2):
            # bf16: both lists of experts give an entry per assignment, so K is split alike
            b = FewMoEBuffers(S, H, D, E, 1, i8=i8, device=DEV)
            c = FewMoEBuffers(S, H, D, 1 if S == 1 or i8 else 2, 1, i8=i8, device=DEV)
            ws = few if S == 1 or i8 else [torch.cat([w, w]) for w in few]
            o = b.forward(x[:S], *many, topk_ids=last[:S], topk_weights=wts[:S])
            r = c.forward(x[:S], *ws, topk_ids=first[:S], topk_weights=wts[:S])
            assert bool(o.any()) and torch.equal(o, r), (i8, S)


@pytest.mark.parametrize("kind", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("S,H,D,E,k,Ds", [(128, 272, 144, 4, 4, 0), (96, 144, 272, 9, 8, 48),
                                          (128, 2048, 48, 3, 3, 0)])
def test_routed_lists_captured(S, H, D, E, k, Ds, kind):
    """More than 256 assignments, an expert's rounds shared by several workgroups: the experts'
    lists of rows are built in any order, the result is the same every time."""
    print(f"[lists S={S} H={H} D={D} E={E} k={k} Ds={Ds} {kind}]", flush=True)
    g = gen(23)
    ly = Layer(g, kind, H, D, E, Ds)
    x, wr = normal(g, (S, H), 1.0, ly.t), normal(g, (H, E), 0.05, ly.t)
    mk = lambda: FewMoEBuffers(S, H, D, E, k, D_shared=Ds, i8=kind == "i8", device=DEV,
                               dtype=moe.MOE_F32 if kind == "f32" else moe.MOE_BF16)
    b, cap = mk(), mk()
    o = b.run(x, wr, *ly.args).clone()
    ref, e = layer_ref(ly, x, b.topk_ids, b.topk_weights)
    check("o", o, ref, e + half(o.dtype) * (ref.abs() + e))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap.run(x, wr, *ly.args)
    for rep in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cap.O, o) and torch.equal(b.run(x, wr, *ly.args), o), rep
