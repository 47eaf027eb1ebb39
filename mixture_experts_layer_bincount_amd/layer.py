"""MoELayer: device buffers plus one moe_forward call per batch.

The layer of the adv12 MoE + EPLB tutorial §4.1 (MoELayer(d_model,
num_experts, top_k) returning the output and the per-expert load), holding
caller-provided device weights.  All compute happens in the HIP library.
"""
from __future__ import annotations

import torch

from . import (DT_BF16, DT_F32, DT_FP8_E4M3, DT_INT4, DT_INT8, LINEAR_BIAS, SWIGLU,
               adapter_workspace, few_workspace, make_adapter_shape, make_shape, make_weights,
               moe_adapter_linear, moe_forward, moe_forward_few, moe_pack_router,
               moe_router_packed_bytes, moe_workspace_bytes)


class MoELayer:
    """Forward pass of one MoE FFN layer on the current HIP device.

    weights: dict of device tensors named as in moe.h (W1, W3, W2 [, s1, s3,
    s2] [, W1s, W3s, W2s [, s1s, s3s, s2s]] for SwiGLU; W, b for Linear+bias).
    overflow: "drop", "reroute" (with reroute_rounds rounds) or "shared", the
    fate of assignments past the capacity.  n_groups / topk_groups: group-
    limited routing (each token uses at most topk_groups groups).  combine:
    "auto", "grouped" or "fused", the form of the combine (moe_combine_form).
    hidden_split: the compensated hidden activation (moe_shape.hidden_split).
    pack_router: split the router's gate once at construction (moe_pack_router)
    instead of in every forward, where the router takes packed weights.
    few: run moe_forward_few (T up to FEW_MAX_TOKENS) instead of moe_forward: fp32's
    precision of the hidden activation and equal bits, faster for narrow or quantised
    experts up to 16 tokens, slower for wide bf16 ones and from 17 tokens on.
    adapters: dict of device tensors A [n, rank, d], B [n, d, rank] (bf16), scales
    [n] fp32 and optionally ranks [n] int32: low-rank adapters in parallel to a
    SwiGLU layer (moe_adapter_linear), added to y row by row as forward's
    adapter_idx says.
    """

    def __init__(self, T, d, E, top_k, d_ff, *, W_g, b_g=None, weights, capacity=-1,
                 kind="swiglu", w_dtype="bf16", has_shared=False, overflow="drop",
                 reroute_rounds=0, n_groups=0, topk_groups=0, combine="auto", hidden_split=False,
                 pack_router=True, few=False, adapters=None, device="cuda"):
        self.kind = SWIGLU if kind == "swiglu" else LINEAR_BIAS
        act = DT_BF16 if self.kind == SWIGLU else DT_F32
        wdt = {"bf16": DT_BF16, "fp8_e4m3": DT_FP8_E4M3, "int8": DT_INT8, "int4": DT_INT4,
               "f32": DT_F32}[w_dtype]
        shape = make_shape(T, d, E, top_k, d_ff, capacity, act, wdt, self.kind, has_shared,
                           overflow, reroute_rounds, n_groups, topk_groups, combine, hidden_split)
        dev = torch.device(device)
        self.W_g = W_g
        self.W_g_packed = None
        if pack_router and moe_router_packed_bytes(shape) > 0:
            # the router's gate split once here, not in every forward
            self.W_g_packed = torch.empty(moe_router_packed_bytes(shape), dtype=torch.uint8,
                                          device=dev)
            moe_pack_router(shape, W_g, self.W_g_packed)
            shape.router_packed = 1
        self.shape = shape
        self.b_g = b_g
        self.weights = make_weights(**weights)
        self.few = bool(few)
        if self.few:
            self.ws = few_workspace(self.shape, dev)
        else:
            self.ws = torch.empty(max(moe_workspace_bytes(self.shape), 256), dtype=torch.uint8,
                                  device=dev)
        self.y = torch.empty((T, d), dtype=torch.float32, device=dev)
        self.topk_idx = torch.empty((T, top_k), dtype=torch.int32, device=dev)
        self.topk_w = torch.empty((T, top_k), dtype=torch.float32, device=dev)
        self.counts = torch.empty((E,), dtype=torch.int32, device=dev)
        self.offsets = torch.empty((E + 1,), dtype=torch.int32, device=dev)
        self.adapters = None
        if adapters is not None:
            if self.kind != SWIGLU:
                raise ValueError("adapters need a SwiGLU layer (bf16 x)")
            n, rank = adapters["A"].shape[:2]
            if tuple(adapters["A"].shape) != (n, rank, d) or \
                    tuple(adapters["B"].shape) != (n, d, rank):
                raise ValueError("adapters: A is [n, rank, d] and B [n, d, rank]")
            if adapters["A"].dtype != torch.bfloat16 or adapters["B"].dtype != torch.bfloat16:
                raise ValueError("adapters: A and B are bf16")
            if tuple(adapters["scales"].shape) != (n,) or \
                    adapters["scales"].dtype != torch.float32:
                raise ValueError("adapters: scales is fp32 [n]")
            ranks = adapters.get("ranks")
            if ranks is not None and (tuple(ranks.shape) != (n,) or ranks.dtype != torch.int32):
                raise ValueError("adapters: ranks is int32 [n]")
            if any(t is not None and t.device.type != dev.type for t in adapters.values()):
                raise ValueError(f"adapters: the tensors lie on the layer's device ({dev.type})")
            self.adapters = dict(adapters)
            self.adapter_shape = make_adapter_shape(T, d, d, n, rank, y_dtype=DT_F32)
            self.adapter_ws = adapter_workspace(self.adapter_shape, dev)

    def forward(self, x: torch.Tensor, stream=None, adapter_idx=None) -> torch.Tensor:
        if adapter_idx is not None:
            if self.adapters is None:
                raise ValueError("adapter_idx needs a layer with adapters")
            if tuple(adapter_idx.shape) != (self.shape.T,) or adapter_idx.dtype != torch.int32:
                raise ValueError("adapter_idx is int32 [T]")
            if adapter_idx.device.type != self.y.device.type:
                raise ValueError("adapter_idx lies on the layer's device")
        W_g = self.W_g_packed if self.W_g_packed is not None else self.W_g
        forward = moe_forward_few if self.few else moe_forward
        forward(self.shape, x, W_g, self.b_g, self.weights, self.y, self.topk_idx,
                self.topk_w, self.counts, self.offsets, self.ws, stream)
        if adapter_idx is not None:
            ad = self.adapters
            moe_adapter_linear(self.adapter_shape, x, None, None, None, ad["A"], ad["B"],
                               ad.get("ranks"), ad["scales"], adapter_idx, self.y, self.y,
                               self.adapter_ws, stream)
        return self.y

    __call__ = forward
