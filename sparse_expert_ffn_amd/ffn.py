"""Binding of include/moe_ffn.h: layer norm, the dense gated feed-forward block
and products with 4-bit weights, with the names of the C ABI.

As the layer's binding it only marshals arguments, but it takes device tensors
only (sizes come from them) and checks their types, shapes, contiguity and
device before the call (ValueError / TypeError; the library's own refusals are
MoeError). A call runs on the tensors' device, on ``stream`` or, if that is
None, on torch's current stream of that device.
"""
from __future__ import annotations

import ctypes

import torch

from . import (MOE_BF16, MOE_F32, MOE_OUTPUT_F32, _check, _stream, _ws, load_library, moe_shape)

__all__ = ["moe_ffn_shape", "make_ffn_shape", "moe_layernorm_forward",
           "moe_layernorm_backward_workspace_bytes", "moe_layernorm_backward",
           "moe_ffn_forward_workspace_bytes", "moe_ffn_forward",
           "moe_ffn_backward_workspace_bytes", "moe_ffn_backward", "moe_w4_weight_bytes",
           "moe_quantize_w4", "moe_pack_w4_weights", "moe_w4_matvec",
           "moe_w4_forward_workspace_bytes", "moe_w4_forward"]

# names of the entry points declared in include/moe_ffn.h
FFN_EXPORTS = tuple(n for n in __all__ if n not in ("moe_ffn_shape", "make_ffn_shape"))


class moe_ffn_shape(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int64), ("H", ctypes.c_int64), ("D", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]

    def __repr__(self):
        return ("moe_ffn_shape(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_)
                + ")")


def make_ffn_shape(S, H, D, dtype=MOE_BF16, out_f32=False) -> moe_ffn_shape:
    return moe_ffn_shape(S, H, D, dtype, MOE_OUTPUT_F32 if out_f32 else 0)


def bind(lib) -> None:
    """Argument types of the entry points in ``lib`` (those it has: a library
    of an earlier build may lack some)."""
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    fp, sp = ctypes.POINTER(moe_ffn_shape), ctypes.POINTER(moe_shape)
    sig = {
        "moe_layernorm_forward": [i64, i64, i32, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp],
        "moe_layernorm_backward_workspace_bytes": [i64, i64, i32],
        "moe_layernorm_backward": [i64, i64, i32] + [vp] * 9 + [sz, vp],
        "moe_ffn_forward_workspace_bytes": [fp],
        "moe_ffn_forward": [fp] + [vp] * 8 + [sz, vp],
        "moe_ffn_backward_workspace_bytes": [fp],
        "moe_ffn_backward": [fp] + [vp] * 12 + [sz, vp],
        "moe_w4_weight_bytes": [i64, i64, i64, i32],
        "moe_quantize_w4": [vp, i64, i64, i64, i32, i32, vp, vp, vp],
        "moe_pack_w4_weights": [vp, vp, i64, i64, i64, i32, vp, vp],
        "moe_w4_matvec": [i64, i64, i64, i64, i32, i32, vp, vp, vp, vp, vp],
        "moe_w4_forward_workspace_bytes": [sp],
        "moe_w4_forward": [sp, i32] + [vp] * 11 + [sz, vp],
    }
    for name, args in sig.items():
        if hasattr(lib, name):
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = sz if name.endswith("_bytes") else ctypes.c_int


def _types(dtype):
    return {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16}.get(dtype)


class _Args:
    """The tensors of one call: checks each, keeps their common device."""

    __slots__ = ("call", "device")

    def __init__(self, call):
        self.call = call
        self.device = None

    def __call__(self, name, t, shape=None, dtype=None, optional=False):
        """Address of a contiguous device tensor (None for an absent optional one)."""
        if t is None and optional:
            return None
        # one test for the usual case (decode calls take a few microseconds in all)
        if (type(t) is torch.Tensor and t.is_cuda and (dtype is None or t.dtype == dtype)
                and (shape is None or t.shape == shape) and t.is_contiguous()):
            d = t.get_device()
            if d == self.device or self.device is None:
                self.device = d
                return t.data_ptr() or None
        return self.refuse(name, t, shape, dtype)

    def refuse(self, name, t, shape, dtype):
        if t is None:
            raise TypeError(f"{self.call}: {name} is required")
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{self.call}: {name} must be a tensor, not {type(t).__name__}")
        if t.device.type != "cuda":
            raise ValueError(f"{self.call}: {name} is on {t.device}: the library takes device "
                             "memory")
        if self.device is not None and t.get_device() != self.device:
            raise ValueError(f"{self.call}: {name} is on {t.device}, others on "
                             f"cuda:{self.device}")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{self.call}: {name} is {t.dtype}, not {dtype}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{self.call}: {name} is {tuple(t.shape)}, not {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{self.call}: {name} must be contiguous")
        self.device = t.get_device()  # a subclass of Tensor
        return t.data_ptr() or None

    def workspace(self, ws):
        if isinstance(ws, tuple):
            return _ws(ws)
        return self("workspace", ws, optional=True), 0 if ws is None else ws.nbytes

    def run(self, stream, check, *args):
        """The call on the tensors' device, its status checked."""
        d = self.device
        f = getattr(load_library(), self.call)
        st = _raw_stream(d) if stream is None else _stream(stream)
        if d == torch.cuda.current_device():
            code = f(*args, st)
        else:
            with torch.cuda.device(d):
                code = f(*args, st)
        if check and code:
            _check(self.call, code)
        return code


# the current stream's handle of a device, without a Stream object where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _matrix(call, name, t):
    if getattr(t, "dim", lambda: 0)() != 2:
        raise ValueError(f"{call}: {name} must be a matrix")
    return t.shape


def _float_dtype(call, name, t):
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise ValueError(f"{call}: {name} is {t.dtype}, not float32 or bfloat16")


# ---------------------------------------------------------------- layer norm

def moe_layernorm_forward(X, gamma, beta, eps, Y, mean=None, rstd=None, stream=None,
                          check=True) -> int:
    """Y = layer norm of the rows of X [S][H]; gamma and beta [H] or None; mean
    and rstd [S] float32, kept for the backward pass, or None."""
    a = _Args("moe_layernorm_forward")
    S, H = _matrix(a.call, "X", X)
    dt = _float_dtype(a.call, "X", X)
    return a.run(stream, check, S, H, dt, a("X", X),
                 a("gamma", gamma, (H,), X.dtype, optional=True),
                 a("beta", beta, (H,), X.dtype, optional=True), eps,
                 a("Y", Y, X.shape, X.dtype),
                 a("mean", mean, (S,), torch.float32, optional=True),
                 a("rstd", rstd, (S,), torch.float32, optional=True))


def moe_layernorm_backward_workspace_bytes(S: int, H: int, dtype: int = MOE_BF16) -> int:
    return int(load_library().moe_layernorm_backward_workspace_bytes(S, H, dtype))


def moe_layernorm_backward(dY, X, gamma, mean, rstd, dX, dgamma, dbeta, workspace, stream=None,
                           check=True) -> int:
    """dX [S][H], and dgamma and dbeta [H] float32 (or None for both)."""
    a = _Args("moe_layernorm_backward")
    S, H = _matrix(a.call, "X", X)
    dt = _float_dtype(a.call, "X", X)
    f32 = torch.float32
    args = [S, H, dt, a("dY", dY, X.shape, X.dtype), a("X", X),
            a("gamma", gamma, (H,), X.dtype, optional=True), a("mean", mean, (S,), f32),
            a("rstd", rstd, (S,), f32), a("dX", dX, X.shape, X.dtype),
            a("dgamma", dgamma, (H,), f32, optional=True),
            a("dbeta", dbeta, (H,), f32, optional=True)]
    wa, wn = a.workspace(workspace)
    return a.run(stream, check, *args, wa, wn)


# ---------------------------------------------------------------- feed-forward block

def moe_ffn_forward_workspace_bytes(shape) -> int:
    return int(load_library().moe_ffn_forward_workspace_bytes(ctypes.byref(shape)))


def moe_ffn_forward(shape, X, W_up, W_gate, W_down, U, G, O, workspace, stream=None,
                    check=True) -> int:
    """O = (SiLU(X W_up) * (X W_gate)) W_down; U and G (the pre-activations) are
    kept for moe_ffn_backward, or None."""
    a = _Args("moe_ffn_forward")
    S, H, D, t = shape.S, shape.H, shape.D, _types(shape.dtype)
    to = torch.float32 if shape.flags & MOE_OUTPUT_F32 else t
    args = [ctypes.byref(shape), a("X", X, (S, H), t), a("W_up", W_up, (H, D), t),
            a("W_gate", W_gate, (H, D), t), a("W_down", W_down, (D, H), t),
            a("U", U, (S, D), t, optional=True), a("G", G, (S, D), t, optional=True),
            a("O", O, (S, H), to)]
    wa, wn = a.workspace(workspace)
    return a.run(stream, check, *args, wa, wn)


def moe_ffn_backward_workspace_bytes(shape) -> int:
    return int(load_library().moe_ffn_backward_workspace_bytes(ctypes.byref(shape)))


def moe_ffn_backward(shape, dO, X, W_up, W_gate, W_down, U, G, dX, dW_up, dW_gate, dW_down,
                     workspace, stream=None, check=True) -> int:
    """Gradients from dO and the kept U and G. dX may be None; the weight
    gradients may be None together."""
    a = _Args("moe_ffn_backward")
    S, H, D, t = shape.S, shape.H, shape.D, _types(shape.dtype)
    tw = torch.float32 if shape.flags & MOE_OUTPUT_F32 else t
    args = [ctypes.byref(shape), a("dO", dO, (S, H), t), a("X", X, (S, H), t),
            a("W_up", W_up, (H, D), t), a("W_gate", W_gate, (H, D), t),
            a("W_down", W_down, (D, H), t), a("U", U, (S, D), t), a("G", G, (S, D), t),
            a("dX", dX, (S, H), t, optional=True), a("dW_up", dW_up, (H, D), tw, optional=True),
            a("dW_gate", dW_gate, (H, D), tw, optional=True),
            a("dW_down", dW_down, (D, H), tw, optional=True)]
    wa, wn = a.workspace(workspace)
    return a.run(stream, check, *args, wa, wn)


# ---------------------------------------------------------------- 4-bit weights

def moe_w4_weight_bytes(E: int, K: int, N: int, group: int) -> int:
    """Bytes of E matrices [K][N] packed for the 4-bit products (0: unsupported)."""
    return int(load_library().moe_w4_weight_bytes(E, K, N, group))


def _ekn(call, name, t):
    if getattr(t, "dim", lambda: 0)() not in (2, 3):
        raise ValueError(f"{call}: {name} must be [E][K][N] or [K][N]")
    return (1,) + tuple(t.shape) if t.dim() == 2 else tuple(t.shape)


def _w4_shapes(call, codes, group):
    E, K, N = _ekn(call, "codes", codes)
    lead = tuple(codes.shape[:-2])
    return E, K, N, lead + (-(-K // max(group, 1)), N)


def moe_quantize_w4(W, group, codes, scales, stream=None, check=True) -> int:
    """Codes (uint8, W's shape) and scales (bfloat16, [.., ceil(K / group), N])
    of a bfloat16 or float32 tensor W [E][K][N] or [K][N]."""
    a = _Args("moe_quantize_w4")
    E, K, N = _ekn(a.call, "W", W)
    dt = _float_dtype(a.call, "W", W)
    return a.run(stream, check, a("W", W), E, K, N, dt, group,
                 a("codes", codes, W.shape, torch.uint8),
                 a("scales", scales, _w4_shapes(a.call, W, group)[3], torch.bfloat16))


def moe_pack_w4_weights(codes, scales, group, packed, stream=None, check=True) -> int:
    """Codes and scales laid out for the products, into ``packed``
    (moe_w4_weight_bytes(E, K, N, group) bytes, uint8)."""
    a = _Args("moe_pack_w4_weights")
    E, K, N, ss = _w4_shapes(a.call, codes, group)
    need = moe_w4_weight_bytes(E, K, N, group)
    return a.run(stream, check, a("codes", codes, dtype=torch.uint8),
                 a("scales", scales, ss, torch.bfloat16), E, K, N, group,
                 a("packed", packed, (need,) if need else None, torch.uint8))


def _w4_weight(call, name, w):
    if not hasattr(w, "packed"):
        raise TypeError(f"{call}: {name} must be a W4Weight, not {type(w).__name__}")


def moe_w4_matvec(X, W, Y, expert_ids=None, stream=None, check=True) -> int:
    """Y = X W for few rows X [S][K] (bfloat16) and a packed weight W
    (layer.W4Weight); Y [S][N] bfloat16 or float32; expert_ids [S] int32: the
    matrix each row takes (none: row of zeros)."""
    a = _Args("moe_w4_matvec")
    _w4_weight(a.call, "W", W)
    S, K = _matrix(a.call, "X", X)
    if K != W.K:
        raise ValueError(f"moe_w4_matvec: X has {K} columns, W {W.K} rows")
    flags = MOE_OUTPUT_F32 if _float_dtype(a.call, "Y", Y) == MOE_F32 else 0
    return a.run(stream, check, S, K, W.N, W.E, W.group, flags, a("X", X, None, torch.bfloat16),
                 a("W", W.packed, (W.nbytes,), torch.uint8),
                 a("expert_ids", expert_ids, (S,), torch.int32, optional=True),
                 a("Y", Y, (S, W.N)))


def moe_w4_forward_workspace_bytes(shape) -> int:
    return int(load_library().moe_w4_forward_workspace_bytes(ctypes.byref(shape)))


def moe_w4_forward(shape, A, W_up, W_gate, W_down, Ws_up, Ws_gate, Ws_down, topk_ids,
                   topk_weights, O, workspace, stream=None, check=True) -> int:
    """The MoE layer's experts with 4-bit weights (layer.W4Weight each, the shared
    expert's None without one) on few tokens, from the router's topk_ids and
    topk_weights."""
    a = _Args("moe_w4_forward")
    S, H, D, Ds, E, k = (shape.S, shape.H, shape.D, shape.D_shared, shape.E, shape.k)
    for name, w in (("W_up", W_up), ("W_gate", W_gate), ("W_down", W_down)):
        _w4_weight(a.call, name, w)
    group = W_up.group

    def packed(name, w, want):
        if w is None:
            return None
        _w4_weight(a.call, name, w)
        if (w.E, w.K, w.N, w.group) != want + (group,):
            raise ValueError(f"{a.call}: {name} is {w}, not {want} in groups of {group}")
        return a(name, w.packed, (w.nbytes,), torch.uint8)

    to = torch.float32 if shape.flags & MOE_OUTPUT_F32 else torch.bfloat16
    args = [ctypes.byref(shape), group, a("A", A, (S, H), torch.bfloat16),
            packed("W_up", W_up, (E, H, D)), packed("W_gate", W_gate, (E, H, D)),
            packed("W_down", W_down, (E, D, H)), packed("Ws_up", Ws_up, (1, H, Ds)),
            packed("Ws_gate", Ws_gate, (1, H, Ds)), packed("Ws_down", Ws_down, (1, Ds, H)),
            a("topk_ids", topk_ids, (S, k), torch.int32),
            a("topk_weights", topk_weights, (S, k), torch.float32), a("O", O, (S, H), to)]
    wa, wn = a.workspace(workspace)
    return a.run(stream, check, *args, wa, wn)
