"""The entry points of include/moe_ffn.h: exported, bound, and refusing bad
arguments on the host (no GPU: each call returns before anything is enqueued)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import sparse_expert_ffn_amd as moe
from sparse_expert_ffn_amd import buildlib, ffn, layer
from sparse_expert_ffn_amd.layer import W4Weight

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = [0x100000 * (i + 1) for i in range(20)]  # distinct aligned addresses, never dereferenced
OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3
BF, F32, MX = moe.MOE_BF16, moe.MOE_F32, moe.MOE_MXFP8


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        moe.build()
    return moe.load_library()


def test_exports_every_declared_symbol(lib):
    text = open(os.path.join(ROOT, "include", "moe_ffn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text))
    assert names == set(moe.FFN_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", moe.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = set(line.split()[-1] for line in out.splitlines() if " T " in line)
    for n in names:
        assert n in exported and getattr(lib, n).argtypes is not None, n
        assert n in moe.__all__ and hasattr(moe, n)
    assert ctypes.sizeof(moe.moe_ffn_shape) == 32


def test_layer_digest_leaves_these_operators_out():
    assert any("ffn" + os.sep in s for s in buildlib.sources())
    before = buildlib.source_digest()
    assert len(before) == 64


def ln_fwd(lib, S=4, H=64, dt=BF, X=A[0], g=A[1], b=A[2], eps=1e-5, Y=A[3], m=A[4], r=A[5]):
    return lib.moe_layernorm_forward(S, H, dt, X, g, b, eps, Y, m, r, None)


def test_layernorm_forward_refusals(lib):
    assert ln_fwd(lib, S=-1) == INVALID
    assert ln_fwd(lib, H=0) == INVALID
    assert ln_fwd(lib, dt=7) == INVALID
    assert ln_fwd(lib, dt=MX) == UNSUPPORTED
    assert ln_fwd(lib, S=2**31) == UNSUPPORTED
    assert ln_fwd(lib, H=2**31) == UNSUPPORTED
    for eps in (-1e-6, float("nan"), float("inf")):
        assert ln_fwd(lib, eps=eps) == INVALID
    assert ln_fwd(lib, m=None) == INVALID          # one of the pair
    assert ln_fwd(lib, X=None) == INVALID
    assert ln_fwd(lib, Y=None) == INVALID
    assert ln_fwd(lib, Y=A[0]) == INVALID          # in place
    assert ln_fwd(lib, X=A[0] + 1) == UNSUPPORTED  # not even an element's alignment
    assert ln_fwd(lib, dt=F32, g=A[1] + 2) == UNSUPPORTED
    assert ln_fwd(lib, m=A[4] + 2) == UNSUPPORTED
    assert ln_fwd(lib, S=0, X=None, Y=None) == OK


def ln_bwd(lib, S=4, H=64, dt=BF, dY=A[0], X=A[1], g=A[2], m=A[3], r=A[4], dX=A[5], dg=A[6],
           db=A[7], ws=A[8], n=1 << 30):
    return lib.moe_layernorm_backward(S, H, dt, dY, X, g, m, r, dX, dg, db, ws, n, None)


def test_layernorm_backward_refusals(lib):
    need = moe.moe_layernorm_backward_workspace_bytes(4, 64)
    assert need > 0
    assert moe.moe_layernorm_backward_workspace_bytes(-1, 64) == 0
    assert moe.moe_layernorm_backward_workspace_bytes(4, 64, MX) == 0
    assert ln_bwd(lib, H=0) == INVALID
    assert ln_bwd(lib, dt=MX) == UNSUPPORTED
    for a in ("dY", "X", "m", "r", "dX"):
        assert ln_bwd(lib, **{a: None}) == INVALID, a
    assert ln_bwd(lib, dg=None) == INVALID
    assert ln_bwd(lib, db=A[6]) == INVALID
    assert ln_bwd(lib, dX=A[1]) == INVALID
    assert ln_bwd(lib, dX=A[0]) == INVALID
    assert ln_bwd(lib, ws=None) == SMALL
    assert ln_bwd(lib, n=need - 1) == SMALL
    assert ln_bwd(lib, ws=A[8] + 4) == UNSUPPORTED
    assert ln_bwd(lib, dX=A[5] + 1) == UNSUPPORTED
    assert ln_bwd(lib, S=0, dY=None, X=None, m=None, r=None, dX=None, dg=None, db=None) == OK


def ffn_fwd(lib, S=16, H=64, D=128, dt=BF, flags=0, X=A[0], Wu=A[1], Wg=A[2], Wd=A[3], U=A[4],
            G=A[5], O=A[6], ws=A[7], n=1 << 40):
    s = moe.moe_ffn_shape(S, H, D, dt, flags)
    return lib.moe_ffn_forward(ctypes.byref(s), X, Wu, Wg, Wd, U, G, O, ws, n, None)


SHAPE_REFUSALS = [(dict(S=-1), INVALID), (dict(H=0), INVALID), (dict(D=0), INVALID),
                  (dict(dt=9), INVALID), (dict(dt=MX), UNSUPPORTED), (dict(flags=2), INVALID),
                  (dict(H=60), UNSUPPORTED), (dict(D=100), UNSUPPORTED),
                  (dict(H=1 << 22), UNSUPPORTED), (dict(S=2**31 - 100), UNSUPPORTED),
                  (dict(S=1 << 26, D=1 << 20), UNSUPPORTED)]


def test_ffn_forward_refusals(lib):
    assert lib.moe_ffn_forward(None, *A[:8], 1 << 40, None) == INVALID
    for kw, code in SHAPE_REFUSALS:
        assert ffn_fwd(lib, **kw) == code, kw
        s = moe.moe_ffn_shape(kw.get("S", 16), kw.get("H", 64), kw.get("D", 128),
                              kw.get("dt", BF), kw.get("flags", 0))
        assert moe.moe_ffn_forward_workspace_bytes(s) == 0
        assert moe.moe_ffn_backward_workspace_bytes(s) == 0
    for a in ("X", "Wu", "Wg", "Wd", "O", "U", "G"):
        assert ffn_fwd(lib, **{a: None}) == INVALID, a
        assert ffn_fwd(lib, **{a: A[12] + 8}) == UNSUPPORTED, a
    for a in ("U", "G", "O", "ws"):
        assert ffn_fwd(lib, **{a: A[0]}) == INVALID, a
    assert ffn_fwd(lib, U=A[6]) == INVALID
    need = moe.moe_ffn_forward_workspace_bytes(moe.make_ffn_shape(16, 64, 128))
    assert need >= 16 * 128 * 2
    assert ffn_fwd(lib, n=need - 1) == SMALL
    assert ffn_fwd(lib, ws=None) == SMALL
    assert ffn_fwd(lib, S=0, X=None, O=None, U=None, G=None) == OK


def ffn_bwd(lib, S=16, H=64, D=128, dt=BF, flags=0, n=1 << 40, **kw):
    s = moe.moe_ffn_shape(S, H, D, dt, flags)
    names = ["dO", "X", "Wu", "Wg", "Wd", "U", "G", "dX", "dWu", "dWg", "dWd", "ws"]
    return lib.moe_ffn_backward(ctypes.byref(s), *[kw.get(a, A[i]) for i, a in enumerate(names)],
                                n, None)


def test_ffn_backward_refusals(lib):
    for kw, code in SHAPE_REFUSALS:
        assert ffn_bwd(lib, **kw) == code, kw
    for a in ("dO", "X", "Wu", "Wg", "Wd", "U", "G", "dWu", "dWg", "dWd"):
        assert ffn_bwd(lib, **{a: None}) == INVALID, a
        assert ffn_bwd(lib, **{a: A[15] + 8}) == UNSUPPORTED, a
    assert ffn_bwd(lib, dX=None, dWu=None, dWg=None, dWd=None) == INVALID  # nothing asked for
    assert ffn_bwd(lib, dX=A[0]) == INVALID
    assert ffn_bwd(lib, dWu=A[9]) == INVALID
    assert ffn_bwd(lib, ws=A[3]) == INVALID
    need = moe.moe_ffn_backward_workspace_bytes(moe.make_ffn_shape(16, 64, 128))
    assert need >= 3 * 16 * 128 * 2
    assert ffn_bwd(lib, n=need - 1) == SMALL
    assert ffn_bwd(lib, ws=None) == SMALL
    none = dict.fromkeys(("dO", "X", "U", "G", "dX", "dWu", "dWg", "dWd"))
    assert ffn_bwd(lib, S=0, **none) == OK


def test_w4_sizes_and_refusals(lib):
    by = moe.moe_w4_weight_bytes
    assert by(1, 128, 16, 128) == 1024 + 32
    assert by(1, 128, 16, 64) == 1024 + 64
    assert by(3, 136, 24, 32) == 3 * 2 * 2 * (1024 + 128)   # tiles filled up
    for bad in ((0, 128, 16, 128), (1, 0, 16, 32), (1, 128, 16, 16), (1, 100, 16, 32),
                (1, 128, 20, 32), (1, 1 << 22, 16, 32), (1 << 17, 128, 16, 32)):
        assert by(*bad) == 0, bad
    q = lambda W=A[0], E=1, K=128, N=16, dt=BF, g=32, c=A[1], s=A[2]: \
        lib.moe_quantize_w4(W, E, K, N, dt, g, c, s, None)
    assert q(g=48) == INVALID and q(dt=MX) == INVALID and q(W=None) == INVALID
    assert q(K=12) == UNSUPPORTED and q(s=A[2] + 1) == UNSUPPORTED
    assert q(E=1 << 16, K=1 << 20, N=1 << 20) == UNSUPPORTED
    p = lambda c=A[0], s=A[1], E=1, K=128, N=16, g=32, o=A[2]: \
        lib.moe_pack_w4_weights(c, s, E, K, N, g, o, None)
    assert p(c=None) == INVALID and p(o=A[0]) == INVALID and p(g=0) == INVALID
    assert p(o=A[2] + 8) == UNSUPPORTED and p(N=4) == UNSUPPORTED


def test_w4_matvec_refusals(lib):
    m = lambda S=1, K=128, N=16, E=1, g=32, f=0, X=A[0], W=A[1], ids=None, Y=A[2]: \
        lib.moe_w4_matvec(S, K, N, E, g, f, X, W, ids, Y, None)
    assert m(S=-1) == INVALID and m(f=2) == INVALID and m(g=33) == INVALID and m(E=0) == INVALID
    assert m(X=None) == INVALID and m(W=None) == INVALID and m(Y=None) == INVALID
    assert m(Y=A[0]) == INVALID
    assert m(K=12) == UNSUPPORTED and m(S=4097) == UNSUPPORTED
    assert m(X=A[0] + 2) == UNSUPPORTED and m(ids=A[3] + 2) == UNSUPPORTED
    assert m(S=4096, K=128, N=(1 << 22) - 8, E=4096, ids=A[3]) == UNSUPPORTED  # too many tiles
    assert m(S=0, X=None, Y=None) == OK


def test_w4_forward_refusals(lib):
    def f(group=32, n=1 << 40, over=None, **kw):
        base = dict(S=4, H=64, D=128, E=8, k=2)
        base.update(kw)
        s = moe.make_shape(**base)
        names = ["A", "Wu", "Wg", "Wd", "Su", "Sg", "Sd", "ids", "w", "O", "ws"]
        a = {x: A[i] for i, x in enumerate(names)}
        if not base.get("D_shared"):
            a.update(Su=None, Sg=None, Sd=None)
        a.update(over or {})
        return lib.moe_w4_forward(ctypes.byref(s), group, *[a[x] for x in names], n, None)

    assert lib.moe_w4_forward(None, 32, *A[:11], 1 << 40, None) == INVALID
    assert f(group=16) == INVALID and f(k=9) == INVALID and f(H=0) == INVALID
    assert f(dtype=7) == INVALID and f(dtype=F32) == UNSUPPORTED and f(dtype=MX) == UNSUPPORTED
    assert f(capacity=4) == UNSUPPORTED and f(atomic_combine=True) == UNSUPPORTED
    assert f(H=60) == UNSUPPORTED and f(D_shared=12) == UNSUPPORTED
    assert f(S=4097) == UNSUPPORTED and f(S=2049) == UNSUPPORTED and f(E=2048) == UNSUPPORTED
    for a in ("A", "Wu", "Wg", "Wd", "ids", "w", "O"):
        assert f(over={a: None}) == INVALID, a
        assert f(over={a: A[15] + 2}) == UNSUPPORTED, a
    assert f(over=dict(Su=A[12])) == INVALID            # shared weights without D_shared
    assert f(D_shared=64, over=dict(Sg=None)) == INVALID
    assert f(over=dict(O=A[0])) == INVALID
    need = moe.moe_w4_forward_workspace_bytes(moe.make_shape(4, 64, 128, 8, 2))
    assert need >= 8 * 128 * 2 + 8 * 64 * 4
    assert f(n=need - 1) == SMALL and f(over=dict(ws=None)) == SMALL
    assert moe.moe_w4_forward_workspace_bytes(moe.make_shape(4, 64, 128, 8, 2, capacity=1)) == 0
    assert f(S=0, over=dict(A=None, O=None, ids=None, w=None)) == OK


def test_an_output_that_is_another_array_is_refused(lib):
    """Two equal pointers, one of them an output's or the workspace's, in every pair."""
    def pairs(call, names, outs):
        for a in outs:
            for b in names:
                if a != b:
                    assert call(**{a: A[14], b: A[14]}) == INVALID, (a, b)

    pairs(lambda **k: ln_fwd(lib, **k), "X g b Y m r".split(), "Y m r".split())
    pairs(lambda **k: ln_bwd(lib, **k), "dY X g m r dX dg db ws".split(), "dX dg db ws".split())
    pairs(lambda **k: ffn_fwd(lib, **k), "X Wu Wg Wd U G O ws".split(), "U G O ws".split())
    pairs(lambda **k: ffn_bwd(lib, **k), "dO X Wu Wg Wd U G dX dWu dWg dWd ws".split(),
          "dX dWu dWg dWd ws".split())

    def quantize(W=A[0], c=A[1], s=A[2]):
        return lib.moe_quantize_w4(W, 1, 128, 16, BF, 32, c, s, None)

    def pack(c=A[0], s=A[1], o=A[2]):
        return lib.moe_pack_w4_weights(c, s, 1, 128, 16, 32, o, None)

    def matvec(X=A[0], W=A[1], ids=A[2], Y=A[3]):
        return lib.moe_w4_matvec(1, 128, 16, 1, 32, 0, X, W, ids, Y, None)

    def layer(**kw):
        s = moe.make_shape(4, 64, 128, 8, 2, 64)
        names = ["A", "Wu", "Wg", "Wd", "Su", "Sg", "Sd", "ids", "w", "O", "ws"]
        return lib.moe_w4_forward(ctypes.byref(s), 32,
                                  *[kw.get(n, A[i]) for i, n in enumerate(names)], 1 << 40, None)

    pairs(quantize, "W c s".split(), "c s".split())
    pairs(pack, "c s o".split(), ["o"])
    pairs(matvec, "X W ids Y".split(), ["Y"])
    pairs(layer, "A Wu Wg Wd Su Sg Sd ids w O ws".split(), "O ws".split())


def test_sizes_past_a_launch_are_refused(lib):
    assert ln_fwd(lib, H=1 << 27) == UNSUPPORTED
    assert ln_bwd(lib, S=1, H=1 << 27) == UNSUPPORTED
    assert moe.moe_layernorm_backward_workspace_bytes(1, 1 << 27, F32) == 0
    wide = dict(S=16, H=1 << 21, D=1 << 21)   # H x D gradients of 2^30 tiles
    assert ffn_bwd(lib, **wide) == UNSUPPORTED
    assert moe.moe_ffn_backward_workspace_bytes(moe.make_ffn_shape(**wide)) == 0


def test_binding_names_a_missing_weight():
    x = torch.zeros(4, 64)
    with pytest.raises(TypeError, match="W must be a W4Weight"):
        moe.moe_w4_matvec(x, None, x)
    with pytest.raises(TypeError, match="W_up must be a W4Weight"):
        moe.moe_w4_forward(moe.make_shape(4, 64, 128, 8, 2), x, None, None, None, None, None,
                           None, x, x, x, None)
    with pytest.raises(ValueError, match="group"):
        W4Weight.quantize(x, group=0)


def test_binding_refuses_bad_tensors():
    """Host tensors, wrong types, shapes and strides are refused before the library."""
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="device memory"):
        moe.moe_layernorm_forward(x, None, None, 1e-5, x.clone())
    with pytest.raises(ValueError, match="matrix"):
        moe.moe_layernorm_forward(x[0], None, None, 1e-5, x)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        moe.moe_layernorm_forward(x.half(), None, None, 1e-5, x)
    a = ffn._Args("call")
    with pytest.raises(TypeError, match="required"):
        a("X", None)
    with pytest.raises(TypeError, match="tensor"):
        a("X", 4096)
    m = torch.empty((4, 8), device="meta")
    with pytest.raises(ValueError, match="device memory"):
        a("X", m)


class _Streams:
    """Stands in for torch's streams and allocations: which stream is current when memory
    is taken and when a call is made, and which streams a tensor's memory waits for."""

    def __init__(self, monkeypatch):
        self.current, self.calls = "reader", []
        outer = self

        class Context:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                self.before = outer.current
                if self.stream is not None:
                    outer.current = self.stream

            def __exit__(self, *exc):
                outer.current = self.before

        class Tensor:
            def __init__(self, shape, owner):
                self.shape, self.owner, self.recorded, self.device = shape, owner, set(), "cuda:0"

            def dim(self):
                return len(self.shape)

            def record_stream(self, stream):
                self.recorded.add(stream)

        self.tensor = lambda *shape: Tensor(shape, self.current)
        monkeypatch.setattr(torch.cuda, "stream", Context)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: self.current)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: f"stream {h}")
        monkeypatch.setattr(torch, "empty", lambda shape, **kw: Tensor(
            shape if isinstance(shape, tuple) else (shape,), self.current))
        for name in ("moe_quantize_w4", "moe_pack_w4_weights"):
            monkeypatch.setattr(layer, name, lambda *a, name=name: self.calls.append((name, a)))


@pytest.mark.parametrize("stream", ["side", 77, None])
def test_packed_weight_belongs_to_the_stream_that_writes_it(lib, monkeypatch, stream):
    """W4Weight from codes and from a tensor: what is allocated on the way comes from the
    pool of the stream that writes it (another stream's work may still use a block of the
    current one's), and no argument, nor the result, is given back to a pool while one of
    the two streams uses it."""
    s = _Streams(monkeypatch)
    on = {"side": "side", 77: "stream 77", None: "reader"}[stream]
    codes, scales = s.tensor(2, 64, 16), s.tensor(2, 2, 16)
    w = W4Weight(codes, scales, 32, stream=stream)
    assert w.packed.owner == on and s.current == "reader"
    if stream is not None:
        assert codes.recorded == scales.recorded == {on} and w.packed.recorded == {"reader"}
    W = s.tensor(2, 64, 16)
    s.calls.clear()
    w = W4Weight.quantize(W, 32, stream=stream)
    assert [n for n, _ in s.calls] == ["moe_quantize_w4", "moe_pack_w4_weights"]
    assert all(t.owner == on for t in (*s.calls[0][1][2:4], w.packed))
    assert s.current == "reader"
    if stream is not None:
        assert W.recorded == {on} and w.packed.recorded == {"reader"}


@pytest.mark.parametrize("current", [0, 1])
def test_router_and_experts_run_on_the_buffers_device(lib, monkeypatch, current):
    """W4MoEBuffers whose device is not the current one: both of the layer's calls are
    made on it (they take the current stream of the device that they run on)."""
    device, calls = [current], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, device[0] = device[0], self.index

        def __exit__(self, *exc):
            device[0] = self.before

    class Tensor:
        def __init__(self, shape, dtype):
            self.shape, self.dtype, self.is_cuda, self.nbytes = shape, dtype, True, 1 << 20

        def get_device(self):
            return 1

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return A[0]

    class Lib:
        def moe_w4_forward(self, *args):
            calls.append(("experts", device[0], args[-1]))
            return 0

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: device[0])
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: Tensor(
        shape if isinstance(shape, tuple) else (shape,), dtype))
    b = layer.W4MoEBuffers(4, 64, 128, 8, 2, group=32, device="cuda:1")
    w = [W4Weight.__new__(W4Weight) for _ in range(3)]
    for v, (K, N) in zip(w, ((64, 128), (64, 128), (128, 64))):
        v.E, v.K, v.N, v.group, v.nbytes = 8, K, N, 32, 64
        v.packed = Tensor((64,), torch.uint8)
    monkeypatch.setattr(torch, "Tensor", Tensor)
    monkeypatch.setattr(ffn, "load_library", Lib)
    monkeypatch.setattr(ffn, "_raw_stream", lambda d: f"stream of {d}")
    monkeypatch.setattr(layer, "moe_gate_topk", lambda *a: calls.append(("router", device[0])))
    x = Tensor((4, 64), torch.bfloat16)
    assert b.run(x, x, *w) is b.O
    assert calls == [("router", 1), ("experts", 1, "stream of 1")] and device[0] == current
    calls.clear()
    b.route(logits_in=x)
    assert calls == [("router", 1)]


def test_layer_digest_follows_the_layers_code_only(tmp_path, monkeypatch):
    """On a copy of the sources: code of the operators in csrc/ffn/ and of moe_ffn.h does not
    change the digest that the layer's counter records carry, the layer's own does."""
    pkg = tmp_path / os.path.basename(buildlib.PKG)
    shutil.copytree(os.path.join(buildlib.PKG, "csrc"), pkg / "csrc")
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    before = buildlib.source_digest()
    monkeypatch.setattr(buildlib, "PKG", str(pkg))
    monkeypatch.setattr(buildlib, "ROOT", str(tmp_path))
    assert buildlib.source_digest() == before

    def edit(path):
        path.write_text(path.read_text() + "\nint added;\n")
        return buildlib.source_digest()

    mine = sorted((pkg / "csrc" / "ffn").iterdir())
    assert any(f.name == "w4.hip" for f in mine)
    for f in (*mine, tmp_path / "include" / "moe_ffn.h"):
        assert edit(f) == before, f.name
    for f in (*sorted(f for f in (pkg / "csrc").iterdir() if f.is_file()),
              tmp_path / "include" / "moe.h"):
        after = edit(f)
        assert after != before, f.name
        before = after
