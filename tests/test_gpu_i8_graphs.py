"""Captured calls of the 8-bit and few-token operators: rows whose codes take more LDS than a
kernel has by default, and graphs that share one workspace."""
import pytest
import torch

from sparse_expert_ffn_amd.layer import I8LinearBuffers, I8Weight
from tests.ffn_util import DEV, gen, normal
from tests.test_gpu_few import KINDS, Layer, buffers
from tests.test_gpu_i8 import weight

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def captured(step):
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    return graph


@pytest.mark.parametrize("S,K,N,out_f32", [(16, 7168, 264, False), (7, 16384, 24, True)])
def test_long_rows_captured_first(S, K, N, out_f32):
    """The first call with such rows is the captured one."""
    g = gen(50)
    x, w = normal(g, (S, K), 1.0, BF), I8Weight(*weight(g, K, N))
    a, b = (I8LinearBuffers(S, K, N, out_f32=out_f32, device=DEV) for _ in range(2))
    graph = captured(lambda: a.run(x, w))
    x0 = x.clone()
    for rep in range(4):
        x.copy_(x0.roll(rep, 0) * (rep + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.Y, b.run(x, w)), rep


@pytest.mark.parametrize("kind", list(KINDS))
def test_graphs_on_one_workspace(kind):
    """A graph of one token and one of 40, in turn, on the same workspace."""
    g = gen(51)
    H, D, E, k, Ds = 528, 144, 16, 4, 48
    ly = Layer(g, kind, H, D, E, Ds)
    wr = normal(g, (H, E), 0.1, ly.t)
    xs = [normal(g, (S, H), 1.0, ly.t) for S in (1, 40)]
    bs, eager = ([buffers(kind, S, H, D, E, k, Ds) for S in (1, 40)] for _ in range(2))
    bs[0].ws = bs[1].ws = max((b.ws for b in bs), key=torch.Tensor.numel)
    graphs = [captured(lambda b=b, x=x: b.run(x, wr, *ly.args)) for b, x in zip(bs, xs)]
    for rep in range(4):
        for x in xs:
            x.mul_(-1.5 if rep % 2 else 0.5)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for b, e, x in zip(bs, eager, xs):
            e.run(x, wr, *ly.args)
            assert torch.equal(b.O, e.O) and torch.equal(b.topk_ids, e.topk_ids), rep
