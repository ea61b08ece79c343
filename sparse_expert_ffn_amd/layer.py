"""Device buffers for one layer shape, and the C-ABI calls in order: the MoE
layer (MoEBuffers), its experts with 4-bit weights (W4MoEBuffers), the dense
gated feed-forward block (FFNBuffers) and layer norm (LayerNormBuffers), the last
two with their backward passes.

Allocation (torch, device memory) happens once in the constructor; ``run``,
``forward`` and ``backward`` only enqueue the library's calls on the stream, so
repeated calls allocate nothing. Outputs are the object's own buffers and hold
until its next call.
"""
from __future__ import annotations

import torch

from . import (MOE_BF16, MOE_F32, MOE_MXFP8, make_ffn_shape, make_shape, moe_align_block_size,
               moe_align_workspace_bytes, moe_ffn_backward, moe_ffn_backward_workspace_bytes,
               moe_ffn_forward, moe_ffn_forward_workspace_bytes, moe_forward,
               moe_forward_workspace_bytes, moe_gate_topk, moe_gate_workspace_bytes,
               moe_layernorm_backward, moe_layernorm_backward_workspace_bytes,
               moe_layernorm_forward, moe_pack_w4_weights, moe_quantize_w4, moe_w4_forward,
               moe_w4_forward_workspace_bytes, moe_w4_weight_bytes)


class MoEBuffers:
    def __init__(self, S, H, D, E, k, D_shared=0, capacity=0, block_size=128, renormalize=1,
                 dtype=MOE_BF16, out_f32=False, atomic_combine=False, sched_quota=False,
                 fused_launch=False, device="cuda", extra_flags=0):
        self.shape = make_shape(S, H, D, E, k, D_shared, capacity, block_size, renormalize,
                                dtype, out_f32, atomic_combine, sched_quota, fused_launch,
                                extra_flags)
        self.tdtype = torch.bfloat16 if dtype != MOE_F32 and not out_f32 else torch.float32
        dev = torch.device(device)
        cap = S * k + E * (block_size - 1)
        i32, f32 = torch.int32, torch.float32
        self.logits = torch.empty((S, E), dtype=f32, device=dev)
        self.topk_ids = torch.empty((S, k), dtype=i32, device=dev)
        self.topk_weights = torch.empty((S, k), dtype=f32, device=dev)
        self.sorted_ids = torch.empty(max(cap, 1), dtype=i32, device=dev)
        self.expert_ids = torch.empty(max(cap // block_size, 1), dtype=i32, device=dev)
        self.ntpp = torch.empty(1, dtype=i32, device=dev)
        self.expert_counts = torch.empty(E, dtype=i32, device=dev)
        gate_ws = moe_gate_workspace_bytes(self.shape)
        self.gate_ws = torch.empty(gate_ws, dtype=torch.uint8, device=dev) if gate_ws else None
        self.align_ws = torch.empty(max(moe_align_workspace_bytes(self.shape), 1),
                                    dtype=torch.uint8, device=dev)
        self.forward_ws = torch.empty(max(moe_forward_workspace_bytes(self.shape), 1),
                                      dtype=torch.uint8, device=dev)
        self.O = torch.empty((S, H), dtype=self.tdtype, device=dev)

    def route(self, A=None, W_router=None, router_bias=None, logits_in=None, stream=None):
        moe_gate_topk(self.shape, A, W_router, router_bias, logits_in, self.logits,
                      self.topk_ids, self.topk_weights, self.gate_ws, stream)
        moe_align_block_size(self.shape, self.topk_ids, self.sorted_ids, self.expert_ids,
                             self.ntpp, self.expert_counts, self.align_ws, stream)

    def forward(self, A, W_up, W_gate, W_down, Ws_up=None, Ws_gate=None, Ws_down=None,
                stream=None):
        moe_forward(self.shape, A, W_up, W_gate, W_down, Ws_up, Ws_gate, Ws_down,
                    self.topk_weights, self.sorted_ids, self.expert_ids, self.ntpp, self.O,
                    self.forward_ws, stream)
        return self.O

    def run(self, A, W_router, W_up, W_gate, W_down, Ws_up=None, Ws_gate=None, Ws_down=None,
            router_bias=None, logits_in=None, stream=None):
        """One pass of the whole layer: gate, top-k, align, experts, combine."""
        self.route(A, W_router, router_bias, logits_in, stream)
        return self.forward(A, W_up, W_gate, W_down, Ws_up, Ws_gate, Ws_down, stream)


def suggest_block_size(S: int, k: int, E: int, capacity: int = 0, dtype: int = 1) -> int:
    """Rows per sorted block (vLLM's fused_moe note grows the block with the
    token count: 16 / 32 / 64, larger for prefill). The GEMM kernels skip
    16-row groups that hold only padding, so a block large enough for one
    expert's rows costs little more than their own work and streams that
    expert's weights once: pick the smallest block that holds the expected
    largest expert, taken as 1.25x the mean rows per expert, or the
    capacity when that is smaller (no expert keeps more). 256 for bf16 and
    MXFP8 only; MXFP8 takes 64 at least."""
    mean = S * k / max(E, 1)
    want = 1.25 * mean
    if capacity > 0:
        want = min(want, capacity)
    top = 256 if dtype != MOE_F32 else 128
    # the MXFP8 tiles come in 64, 128 and 256 rows
    for bm in ((64, 128, 256) if dtype == MOE_MXFP8 else (16, 32, 64, 128, 256)):
        if bm >= want or bm == top:
            return bm
    return top


def _dtype(dtype):
    if dtype not in (MOE_F32, MOE_BF16):
        raise ValueError("dtype must be MOE_F32 or MOE_BF16")
    return torch.float32 if dtype == MOE_F32 else torch.bfloat16


class LayerNormBuffers:
    """Layer norm over [S][H], forward and backward."""

    def __init__(self, S, H, dtype=MOE_BF16, device="cuda"):
        t, f32 = _dtype(dtype), torch.float32
        self.Y = torch.empty((S, H), dtype=t, device=device)
        self.mean = torch.empty(S, dtype=f32, device=device)
        self.rstd = torch.empty(S, dtype=f32, device=device)
        self.dX = torch.empty((S, H), dtype=t, device=device)
        self.dgamma = torch.empty(H, dtype=f32, device=device)
        self.dbeta = torch.empty(H, dtype=f32, device=device)
        self.ws = torch.empty(moe_layernorm_backward_workspace_bytes(S, H, dtype),
                              dtype=torch.uint8, device=device)

    def forward(self, X, gamma=None, beta=None, eps=1e-5, stream=None):
        moe_layernorm_forward(X, gamma, beta, eps, self.Y, self.mean, self.rstd, stream)
        return self.Y

    def backward(self, dY, X, gamma=None, mean=None, rstd=None, stream=None):
        """(dX, dgamma, dbeta); mean and rstd: by default the last forward's."""
        moe_layernorm_backward(dY, X, gamma, self.mean if mean is None else mean,
                               self.rstd if rstd is None else rstd, self.dX, self.dgamma,
                               self.dbeta, self.ws, stream)
        return self.dX, self.dgamma, self.dbeta


class FFNBuffers:
    """The dense gated feed-forward block. keep: the forward pass keeps U and G
    for a backward pass; train: buffers of the backward pass too; out_f32: O and
    the weight gradients are fp32."""

    def __init__(self, S, H, D, dtype=MOE_BF16, keep=True, train=False, out_f32=False,
                 device="cuda"):
        t = _dtype(dtype)
        tf = torch.float32 if out_f32 else t
        self.shape = make_ffn_shape(S, H, D, dtype, out_f32)
        empty = lambda *n, dt=t: torch.empty(n, dtype=dt, device=device)
        self.O = empty(S, H, dt=tf)
        self.U, self.G = (empty(S, D), empty(S, D)) if keep else (None, None)
        ws = moe_ffn_forward_workspace_bytes(self.shape)
        if train:
            self.dX = empty(S, H)
            self.dW_up, self.dW_gate = empty(H, D, dt=tf), empty(H, D, dt=tf)
            self.dW_down = empty(D, H, dt=tf)
            ws = max(ws, moe_ffn_backward_workspace_bytes(self.shape))
        self.ws = empty(ws, dt=torch.uint8)

    def forward(self, X, W_up, W_gate, W_down, stream=None):
        moe_ffn_forward(self.shape, X, W_up, W_gate, W_down, self.U, self.G, self.O, self.ws,
                        stream)
        return self.O

    def backward(self, dO, X, W_up, W_gate, W_down, U=None, G=None, stream=None):
        """(dX, dW_up, dW_gate, dW_down); U and G: by default the last forward's."""
        if not hasattr(self, "dX"):
            raise ValueError("FFNBuffers without train=True have no backward pass")
        moe_ffn_backward(self.shape, dO, X, W_up, W_gate, W_down, self.U if U is None else U,
                         self.G if G is None else G, self.dX, self.dW_up, self.dW_gate,
                         self.dW_down, self.ws, stream)
        return self.dX, self.dW_up, self.dW_gate, self.dW_down


def _as_stream(stream, device):
    """A stream's handle as a Stream; Streams and None as they are."""
    return torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream


class W4Weight:
    """A weight [E][K][N] or [K][N] as 4-bit codes and group scales, packed for the
    products (codes and scales are not kept).

    With a stream, the work runs there, after what it already holds: whoever fills codes
    and scales, or reads the packed weight, on another stream has to order the two. The
    packed weight is allocated on that stream too (a block of the current stream's pool
    may still be in use by its work), and is not reused before the current stream's
    work as of its release; a weight released while a third stream reads it needs
    ``packed.record_stream`` of that one. codes, scales and W may be released at once."""

    def __init__(self, codes, scales, group=128, stream=None):
        self.E, self.K, self.N = (1, *codes.shape) if codes.dim() == 2 else tuple(codes.shape)
        self.group = group
        self.nbytes = moe_w4_weight_bytes(self.E, self.K, self.N, group)
        stream = _as_stream(stream, codes.device)
        with torch.cuda.stream(stream):
            self.packed = torch.empty(self.nbytes, dtype=torch.uint8, device=codes.device)
            moe_pack_w4_weights(codes, scales, group, self.packed, stream)
        if stream is not None:
            codes.record_stream(stream)
            scales.record_stream(stream)
            self.packed.record_stream(torch.cuda.current_stream(codes.device))

    @classmethod
    def quantize(cls, W, group=128, stream=None):
        """The library's quantisation of a bf16 or fp32 tensor."""
        K, N = W.shape[-2:]
        if group < 1:
            raise ValueError(f"W4Weight.quantize: group is {group}, not 32, 64 or 128")
        stream = _as_stream(stream, W.device)
        # the codes and scales are given back when this returns: they belong to the
        # stream that the two calls run on, so that nothing reuses them before
        with torch.cuda.stream(stream):
            codes = torch.empty(W.shape, dtype=torch.uint8, device=W.device)
            scales = torch.empty((*W.shape[:-2], -(-K // group), N), dtype=torch.bfloat16,
                                 device=W.device)
            moe_quantize_w4(W, group, codes, scales, stream)
        if stream is not None:
            W.record_stream(stream)
        return cls(codes, scales, group, stream)

    def __repr__(self):
        return f"W4Weight(E={self.E}, K={self.K}, N={self.N}, group={self.group})"


class W4MoEBuffers:
    """The MoE layer with 4-bit expert weights for few tokens: router, then the
    experts (no align step). The calls run on the buffers' device, on ``stream`` or its
    current stream."""

    def __init__(self, S, H, D, E, k, D_shared=0, group=128, renormalize=1, out_f32=False,
                 device="cuda"):
        self.shape = make_shape(S, H, D, E, k, D_shared, renormalize=renormalize,
                                out_f32=out_f32)
        self.group = group
        f32 = torch.float32
        self.logits = torch.empty((S, E), dtype=f32, device=device)
        self.topk_ids = torch.empty((S, k), dtype=torch.int32, device=device)
        self.topk_weights = torch.empty((S, k), dtype=f32, device=device)
        self.O = torch.empty((S, H), dtype=f32 if out_f32 else torch.bfloat16, device=device)
        gate_ws = moe_gate_workspace_bytes(self.shape)
        self.gate_ws = torch.empty(gate_ws, dtype=torch.uint8, device=device) if gate_ws else None
        self.ws = torch.empty(moe_w4_forward_workspace_bytes(self.shape), dtype=torch.uint8,
                              device=device)

    def route(self, A=None, W_router=None, router_bias=None, logits_in=None, stream=None):
        args = (self.shape, A, W_router, router_bias, logits_in, self.logits, self.topk_ids,
                self.topk_weights, self.gate_ws, stream)
        # the router's binding takes the current device and its stream, the experts' the
        # tensors': both on the buffers' device, so that they are in order
        if self.O.get_device() == torch.cuda.current_device():
            moe_gate_topk(*args)
        else:
            with torch.cuda.device(self.O.get_device()):
                moe_gate_topk(*args)

    def forward(self, A, W_up, W_gate, W_down, Ws_up=None, Ws_gate=None, Ws_down=None,
                topk_ids=None, topk_weights=None, stream=None):
        """The experts; topk_ids and topk_weights: by default the last route's."""
        moe_w4_forward(self.shape, A, W_up, W_gate, W_down, Ws_up, Ws_gate, Ws_down,
                       self.topk_ids if topk_ids is None else topk_ids,
                       self.topk_weights if topk_weights is None else topk_weights, self.O,
                       self.ws, stream)
        return self.O

    def run(self, A, W_router, W_up, W_gate, W_down, Ws_up=None, Ws_gate=None, Ws_down=None,
            router_bias=None, logits_in=None, stream=None):
        """One pass of the whole layer: gate, top-k, experts, combine."""
        self.route(A, W_router, router_bias, logits_in, stream)
        return self.forward(A, W_up, W_gate, W_down, Ws_up, Ws_gate, Ws_down, stream=stream)
