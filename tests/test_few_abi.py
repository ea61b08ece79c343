"""The entry points of the MoE layer for a few tokens: bad arguments are refused on the host
(no GPU: each call returns before anything is enqueued)."""
import ctypes
import os

import pytest

import sparse_expert_ffn_amd as moe

A = [0x100000 * (i + 1) for i in range(20)]  # distinct aligned addresses, never dereferenced
OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3
BF, F32, MX = moe.MOE_BF16, moe.MOE_F32, moe.MOE_MXFP8
NAMES = ["A", "Wr", "bias", "Wu", "Wg", "Wd", "Su", "Sg", "Sd", "ids", "w", "O", "ws"]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        moe.build()
    return moe.load_library()


def shape(S=4, H=64, D=128, E=16, k=2, Ds=32, **kw):
    return moe.make_shape(S, H, D, E, k, Ds, **kw)


def call(f, s, n=1 << 40, **kw):
    return f(ctypes.byref(s), *[kw.get(a, A[i]) for i, a in enumerate(NAMES)], n, None)


SHAPES = [(dict(S=-1), INVALID), (dict(H=0), INVALID), (dict(D=0), INVALID), (dict(E=0), INVALID),
          (dict(k=0), INVALID), (dict(k=17), INVALID), (dict(Ds=-16), INVALID),
          (dict(dtype=7), INVALID), (dict(capacity=-1), INVALID), (dict(dtype=MX), UNSUPPORTED),
          (dict(capacity=4), UNSUPPORTED), (dict(S=129), UNSUPPORTED), (dict(H=68), UNSUPPORTED),
          (dict(D=132), UNSUPPORTED), (dict(Ds=20), UNSUPPORTED), (dict(H=65552), UNSUPPORTED),
          (dict(D=65552), UNSUPPORTED), (dict(E=1025), UNSUPPORTED),
          (dict(E=64, k=33), UNSUPPORTED), (dict(H=65536, D=32768), UNSUPPORTED),
          (dict(H=65536, Ds=32768), UNSUPPORTED), (dict(atomic_combine=True), UNSUPPORTED)]


@pytest.mark.parametrize("i8", [False, True], ids=["plain", "i8"])
def test_shapes(lib, i8):
    f = lib.moe_few_i8_forward if i8 else lib.moe_few_forward
    size = moe.moe_few_i8_workspace_bytes if i8 else moe.moe_few_workspace_bytes
    assert f(None, *A[:13], 1 << 40, None) == INVALID
    for kw, code in SHAPES:
        s = shape(**kw)
        assert call(f, s) == code, kw
        assert size(s) == 0, kw
    assert size(shape()) > 0
    if i8:
        assert call(f, shape(dtype=F32)) == UNSUPPORTED
        assert call(f, shape(H=72)) == UNSUPPORTED and call(f, shape(D=72)) == UNSUPPORTED


@pytest.mark.parametrize("i8", [False, True], ids=["plain", "i8"])
def test_arguments(lib, i8):
    f = lib.moe_few_i8_forward if i8 else lib.moe_few_forward
    size = moe.moe_few_i8_workspace_bytes if i8 else moe.moe_few_workspace_bytes
    s = shape()
    need = size(s)
    for a in ("A", "Wu", "Wg", "Wd", "Su", "Sg", "Sd", "ids", "w", "O"):
        assert call(f, s, **{a: None}) == INVALID, a
    assert call(f, s, Wr=None) == INVALID                       # a bias without a router
    assert call(f, shape(Ds=0)) == INVALID                      # a shared expert without a size
    for a in ("A", "Wr", "Wu", "Wd", "Sg", "O", "ws"):
        assert call(f, s, **{a: A[15] + 8}) == UNSUPPORTED, a
    for a in ("bias", "ids", "w"):
        assert call(f, s, **{a: A[15] + 2}) == UNSUPPORTED, a
    for a in ("O", "ws", "ids", "w"):                           # outputs that are inputs
        for b in ("A", "Wr", "bias", "Wu", "Sd"):
            assert call(f, s, **{a: A[NAMES.index(b)]}) == INVALID, (a, b)
    assert call(f, s, O=A[12]) == INVALID and call(f, s, ids=A[10]) == INVALID
    assert call(f, s, ids=A[11]) == INVALID and call(f, s, w=A[12]) == INVALID
    assert call(f, s, n=need - 1) == SMALL and call(f, s, ws=None) == SMALL
    assert call(f, shape(S=0), A=None, O=None, ids=None) == OK
