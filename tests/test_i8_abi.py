"""The entry points of the 8-bit products: bad arguments are refused on the host (no GPU:
each call returns before anything is enqueued)."""
import ctypes
import os

import pytest

import sparse_expert_ffn_amd as moe

A = [0x100000 * (i + 1) for i in range(20)]  # distinct aligned addresses, never dereferenced
OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3
BF, F32, MX = moe.MOE_BF16, moe.MOE_F32, moe.MOE_MXFP8


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        moe.build()
    return moe.load_library()


# E, K, N
MATRICES = [((0, 64, 16), INVALID), ((1, 0, 16), INVALID), ((1, 64, 0), INVALID),
            ((-1, 64, 16), INVALID), ((1, 72, 16), UNSUPPORTED), ((1, 64, 12), UNSUPPORTED),
            ((1, 131088, 16), UNSUPPORTED), ((1, 64, 1 << 22), UNSUPPORTED),
            ((1 << 17, 64, 16), UNSUPPORTED)]


def test_weights(lib):
    q = lambda ekn, dt=BF, W=A[0], c=A[1], s=A[2]: lib.moe_quantize_i8(W, *ekn, dt, c, s, None)
    p = lambda ekn, c=A[0], s=A[1], o=A[2]: lib.moe_pack_i8_weights(c, s, *ekn, o, None)
    for ekn, code in MATRICES:
        assert moe.moe_i8_weight_bytes(*ekn) == 0
        assert q(ekn) == code and p(ekn) == code, ekn
    assert moe.moe_i8_weight_bytes(3, 80, 24) == 3 * (2 * 2 * 1024 + 2 * 64)
    ok = (1, 64, 16)
    assert q(ok, dt=MX) == INVALID
    for kw in ("W", "c", "s"):
        assert q(ok, **{kw: None}) == INVALID
        assert q(ok, **{kw: A[5] + 2}) == UNSUPPORTED
    assert q(ok, c=A[0]) == INVALID and q(ok, s=A[0]) == INVALID and q(ok, s=A[1]) == INVALID
    for kw in ("c", "s", "o"):
        assert p(ok, **{kw: None}) == INVALID
    assert p(ok, o=A[0]) == INVALID and p(ok, o=A[1]) == INVALID
    assert p(ok, s=A[5] + 2) == UNSUPPORTED and p(ok, o=A[5] + 4) == UNSUPPORTED
    assert q((1 << 16, 64, 1 << 21)) == UNSUPPORTED  # more workgroups than a launch takes


def test_rows(lib):
    r = lambda S=4, K=64, dt=BF, X=A[0], c=A[1], s=A[2]: lib.moe_quantize_i8_rows(
        X, S, K, dt, c, s, None)
    assert r(S=-1) == INVALID and r(K=0) == INVALID and r(dt=MX) == INVALID
    assert r(K=72) == UNSUPPORTED and r(K=131088) == UNSUPPORTED
    assert r(S=1 << 26) == UNSUPPORTED and r(S=1 << 24, K=8192) == UNSUPPORTED
    assert r(S=1 << 22, K=65536) == UNSUPPORTED
    for kw in ("X", "c", "s"):
        assert r(**{kw: None}) == INVALID
        assert r(**{kw: A[5] + 2}) == UNSUPPORTED
    assert r(c=A[0]) == INVALID and r(s=A[0]) == INVALID and r(s=A[1]) == INVALID
    assert r(S=0, X=None, c=None, s=None) == OK


def test_matmul(lib):
    def f(S=4, K=64, N=16, dt=BF, flags=0, X=A[0], rs=None, W=A[1], Y=A[2], ws=A[3], n=1 << 40):
        return lib.moe_i8_matmul(S, K, N, dt, flags, X, rs, W, Y, ws, n, None)
    for (_, K, N), code in MATRICES[1:3] + MATRICES[4:8]:
        assert f(K=K, N=N) == code, (K, N)
        assert moe.moe_i8_matmul_workspace_bytes(4, K, N) == 0
    assert f(S=-1) == INVALID and moe.moe_i8_matmul_workspace_bytes(-1, 64, 16) == 0
    assert f(S=2**31) == UNSUPPORTED and f(S=1 << 26, N=1 << 20) == UNSUPPORTED
    assert f(dt=MX) == INVALID and f(flags=2) == INVALID
    for kw in ("X", "W", "Y"):
        assert f(**{kw: None}) == INVALID
        assert f(**{kw: A[5] + 8}) == UNSUPPORTED
    assert f(rs=A[5] + 2) == UNSUPPORTED
    assert f(Y=A[0]) == INVALID and f(Y=A[1]) == INVALID and f(rs=A[2]) == INVALID
    assert f(ws=A[0]) == INVALID and f(ws=A[2]) == INVALID and f(ws=A[5] + 4) == UNSUPPORTED
    need = moe.moe_i8_matmul_workspace_bytes(4, 64, 16)
    assert need > 0  # few rows are quantised in the product's launch, more before it
    assert moe.moe_i8_matmul_workspace_bytes(4000, 64, 16) >= 4000 * (64 + 4)
    assert f(n=need - 1) == SMALL and f(ws=None) == SMALL
    assert f(S=0, X=None, Y=None) == OK


def test_ffn(lib):
    def f(S=16, H=64, D=128, dt=BF, flags=0, n=1 << 40, **kw):
        s = moe.moe_ffn_shape(S, H, D, dt, flags)
        names = ["X", "Wu", "Wg", "Wd", "O", "ws"]
        return lib.moe_i8_ffn_forward(ctypes.byref(s), *[kw.get(a, A[i]) for i, a in
                                                         enumerate(names)], n, None)
    for kw, code in [(dict(S=-1), INVALID), (dict(H=0), INVALID), (dict(D=0), INVALID),
                     (dict(dt=9), INVALID), (dict(dt=MX), UNSUPPORTED), (dict(flags=2), INVALID),
                     (dict(H=72), UNSUPPORTED), (dict(D=24), UNSUPPORTED),
                     (dict(H=131088), UNSUPPORTED), (dict(D=131088), UNSUPPORTED),
                     (dict(S=2**31 - 100), UNSUPPORTED), (dict(S=1 << 25, D=65536), UNSUPPORTED)]:
        assert f(**kw) == code, kw
        s = moe.moe_ffn_shape(kw.get("S", 16), kw.get("H", 64), kw.get("D", 128),
                              kw.get("dt", BF), kw.get("flags", 0))
        assert moe.moe_i8_ffn_workspace_bytes(s) == 0
    for a in ("X", "Wu", "Wg", "Wd", "O"):
        assert f(**{a: None}) == INVALID, a
        assert f(**{a: A[9] + 8}) == UNSUPPORTED, a
    assert f(O=A[0]) == INVALID and f(O=A[3]) == INVALID and f(ws=A[4]) == INVALID
    need = moe.moe_i8_ffn_workspace_bytes(moe.make_ffn_shape(16, 64, 128))
    assert f(n=need - 1) == SMALL and f(ws=None) == SMALL and f(ws=A[9] + 4) == UNSUPPORTED
    assert f(S=0, X=None, O=None) == OK
