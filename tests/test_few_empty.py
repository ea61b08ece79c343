"""A batch without tokens: every size query answers (in a process of its own, since a division
by zero on the host would end this one), and the buffers' passes return nothing."""
import os
import subprocess
import sys

import pytest
import torch

import sparse_expert_ffn_amd as moe
from sparse_expert_ffn_amd.layer import FewMoEBuffers, I8FFNBuffers, I8LinearBuffers, I8Weight

QUERIES = [f"moe_few{i8}_workspace_bytes(m.make_shape(0, {H}, {D}, {E}, {k}, {Ds}))"
           for i8 in ("", "_i8") for H, D, E, k, Ds in
           ((64, 32, 4, 2, 0), (64, 32, 4, 2, 32), (16, 16, 1, 1, 0), (7168, 2048, 256, 8, 2048),
            (2048, 768, 1024, 32, 0))]
QUERIES += ["moe_few_workspace_bytes(m.make_shape(0, 64, 32, 4, 2, 32, dtype=m.MOE_F32))",
            "moe_i8_matmul_workspace_bytes(0, 64, 32)",
            "moe_i8_ffn_workspace_bytes(m.make_ffn_shape(0, 64, 32))"]


def test_sizes():
    if not os.path.exists(moe.LIB_PATH):
        moe.build()
    code = "import sparse_expert_ffn_amd as m\n"
    code += "\n".join(f"print(m.{q}, flush=True)" for q in QUERIES)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    sizes = r.stdout.split()
    assert r.returncode == 0, (r.returncode, QUERIES[len(sizes)], r.stderr[-500:])
    assert len(sizes) == len(QUERIES) and all(0 < int(n) <= 1024 for n in sizes), sizes


@pytest.mark.gpu
@pytest.mark.parametrize("i8", [False, True], ids=["plain", "i8"])
def test_buffers(i8):
    H, D, E, k, Ds = 64, 32, 4, 2, 16
    bf = dict(dtype=torch.bfloat16, device="cuda")
    if i8:
        w = lambda *n: I8Weight.quantize(torch.ones(n, **bf))
    else:
        w = lambda *n: torch.ones(n, **bf)
    experts = [w(E, H, D), w(E, H, D), w(E, D, H), w(H, Ds), w(H, Ds), w(Ds, H)]
    x, wr = torch.empty((0, H), **bf), torch.ones((H, E), **bf)
    b = FewMoEBuffers(0, H, D, E, k, D_shared=Ds, i8=i8)
    assert b.ws.numel() > 0
    assert b.run(x, wr, *experts).shape == (0, H) and b.topk_ids.shape == (0, k)
    assert b.forward(x, *experts).shape == (0, H)


@pytest.mark.gpu
def test_8bit_buffers():
    bf = dict(dtype=torch.bfloat16, device="cuda")
    up, down = (I8Weight.quantize(torch.ones(n, **bf)) for n in ((64, 32), (32, 64)))
    x = torch.empty((0, 64), **bf)
    assert I8LinearBuffers(0, 64, 32).run(x, up).shape == (0, 32)
    assert I8FFNBuffers(0, 64, 32).forward(x, up, up, down).shape == (0, 64)
