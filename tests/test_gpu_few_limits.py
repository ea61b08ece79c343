"""The MoE layer for a few tokens at its limits. Routing: up to 8 tokens each workgroup selects
for itself (up to 8 x 1024 scores, 256 assignments), beyond a launch does it. Sizes: the largest
H, D and D_shared, where they meet the others."""
import pytest
import torch

from tests.ffn_util import DEV, U, check, gen, half, mm, normal
from tests.test_gpu_few import KINDS, Layer, buffers, layer_ref

pytestmark = pytest.mark.gpu

# several parts of 512 rows of H; E that is and is no whole number of 16-byte vectors
CASES = [(8, 1040, 1024, 32, True, 1), (8, 2064, 256, 8, False, 0), (8, 1040, 256, 32, False, 1),
         (9, 1040, 1024, 32, False, 1), (7, 1040, 1023, 31, True, 0), (1, 7168, 1024, 32, True, 1),
         (8, 528, 500, 7, True, 1), (2, 4112, 1021, 1, False, 0), (3, 4096, 640, 16, False, 1)]


def scores(x, wr, bias):
    """In 64 bits, and how far the kernel's may be: a wave adds 64 rows of H in fp32 in matrix
    instructions, then 8 waves' sums are added, each addition within an ulp (2 u) of what it
    has so far, a product within u; these parts are added in 64 bits and rounded once (u), and
    the bias is added in fp32 (u)."""
    s = mm(x, wr)
    e = (2 * (64 + 8) + 1) * U * mm(x.abs(), wr.abs()) + 1.01 * U * s.abs()
    if bias is not None:
        s = s + bias.double()
        e = e + 1.01 * U * s.abs()
    return s, e


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("S,H,E,k,bias,renorm", CASES)
def test_limits(S, H, E, k, bias, renorm, kind):
    """Each choice, slot by slot, is at least as good as every expert that was not chosen
    before it, to these two experts' own errors; weights and output follow the choices."""
    print(f"[route S={S} H={H} E={E} k={k} {kind}]", flush=True)
    g = gen(40)
    ly = Layer(g, kind, H, 32, E)
    x = normal(g, (S, H), 1.0, ly.t)
    wr = normal(g, (H, E), H ** -0.5, ly.t)
    bs = torch.randn(E, generator=g, device=DEV) if bias else None
    b = buffers(kind, S, H, 32, E, k, renormalize=renorm)
    b.ws.fill_(0xFF)
    o = b.run(x, wr, *ly.args, router_bias=bs)
    ids = b.topk_ids.long()
    assert int(ids.min()) >= 0 and int(ids.max()) < E
    assert all(len(set(r)) == k for r in ids.tolist())
    s, e = scores(x, wr, bs)
    most = s + e
    left = s - e
    for j in range(k):
        at = ids[:, j:j + 1]
        assert bool((torch.gather(most, 1, at) >= left.amax(1, keepdim=True)).all()), j
        left.scatter_(1, at, float("-inf"))
    # exp(s_i - s_0) over a sum of such: off by the scores' errors, in 64 bits, rounded once
    chosen = torch.gather(s, 1, ids)
    top = s.amax(1, keepdim=True)
    den = torch.exp((chosen if renorm else s) - top).sum(1, keepdim=True)
    w = torch.exp(chosen - top) / den
    ew = 1.01 * (torch.gather(e, 1, ids) + e.amax(1, keepdim=True)) + 2 * U
    check("w", b.topk_weights, w, ew * w + 1e-38)
    ref, eo = layer_ref(ly, x, b.topk_ids, b.topk_weights)
    check("o", o, ref, eo + half(o.dtype) * (ref.abs() + eo))


@pytest.mark.parametrize("kind", list(KINDS))
def test_one_token_more(kind):
    """8 tokens routed by each workgroup for itself and the same 8 with a ninth, routed by a
    launch: the same ids, and weights to the bit."""
    g = gen(41)
    H, E, k = 1040, 1024, 32
    ly = Layer(g, kind, H, 16, E)
    x = normal(g, (9, H), 1.0, ly.t)
    wr = normal(g, (H, E), H ** -0.5, ly.t)
    few, many = buffers(kind, 8, H, 16, E, k), buffers(kind, 9, H, 16, E, k)
    few.run(x[:8].contiguous(), wr, *ly.args)
    many.run(x, wr, *ly.args)
    assert torch.equal(few.topk_ids, many.topk_ids[:8])
    assert torch.equal(few.topk_weights, many.topk_weights[:8])


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("S,H,D,E,k,Ds", [(3, 65536, 48, 4, 2, 16), (40, 80, 65536, 2, 2, 0),
                                          (128, 48, 16, 3, 1, 65536), (128, 16, 65536, 32, 32, 0)])
def test_largest_sizes(S, H, D, E, k, Ds, kind):
    print(f"[largest S={S} H={H} D={D} E={E} k={k} Ds={Ds} {kind}]", flush=True)
    g = gen(42)
    ly = Layer(g, kind, H, D, E, Ds)
    x = normal(g, (S, H), 1.0, ly.t)
    wr = normal(g, (H, E), H ** -0.5, ly.t)
    b = buffers(kind, S, H, D, E, k, Ds)
    b.ws.fill_(0xFF)
    o = b.run(x, wr, *ly.args)
    ref, e = layer_ref(ly, x, b.topk_ids, b.topk_weights)
    check("o", o, ref, e + half(o.dtype) * (ref.abs() + e))
