"""One layer from the residual stream: residual addition and norm, the router
and the routed experts, on buffers allocated once.

``RoutedBlock`` runs the calls of ``include/moe.h`` in the order a decoder layer
does: moe_add_rms_norm -> moe_router_logits -> moe_router_topk -> the routed
branch.  With FP8 experts the norm's e4m3 row is what is dispatched
(moe_dispatch_fp8, then the lane's GEMMs and combine), so no later step
quantises; with 4-bit integer experts (up to ``W4_MAX_TOKENS`` tokens) the BF16
row goes to moe_experts_w4, with 4-bit floating-point ones to a 4-bit lane
(moe_dispatch_quant_fp4, both products, combine).  Every call is asynchronous on one stream and can be captured
into a CUDA graph.
"""
from __future__ import annotations

import torch

from . import api

__all__ = ["RoutedBlock"]


class RoutedBlock:
    """``T`` tokens of hidden size ``H``, ``E`` experts of intermediate size
    ``I``, ``K`` per token.  ``norm_weight [H]`` and ``router_weight [E, H]``
    belong to the layer; ``router`` are the options of ``moe_router_topk``
    (``score``, ``bias``, ``groups``, ``topk_groups``, ``group_top``,
    ``renormalize``, ``scale``).  ``capacity`` rows per expert on the FP8 path
    (default: room for every route) in the packed layout; ``w4`` takes the
    4-bit integer path instead, ``fp4`` ("nvfp4" or "mxfp4", with
    ``fp4_gscales`` as of ``MoeLayerBuffers``) the 4-bit floating-point one."""

    def __init__(self, T: int, E: int, K: int, H: int, I: int, norm_weight, router_weight, *,
                 eps: float = 1e-6, capacity: int | None = None, w4: bool = False,
                 fp4: str | None = None, fp4_gscales: tuple = (None, None, None, None), **router):
        d = norm_weight.device
        if w4 and fp4:
            raise ValueError("w4 or fp4, not both")
        self.T, self.E, self.K, self.H, self.I, self.eps, self.w4 = T, E, K, H, I, eps, w4
        self.fp4 = fp4
        self.norm_weight, self.router_weight, self.router = norm_weight, router_weight, router
        self.h = torch.empty(T, H, dtype=torch.bfloat16, device=d)
        self.logits = torch.empty(T, E, dtype=torch.float32, device=d)
        self.topk_idx = torch.empty(T, K, dtype=torch.int32, device=d)
        self.topk_w = torch.empty(T, K, dtype=torch.float32, device=d)
        self.router_status = torch.zeros(2, dtype=torch.int32, device=d)
        self.hq = self.hs = self.lane = self.workspace = None
        if w4:
            if T > api.W4_MAX_TOKENS:
                raise ValueError(f"4-bit experts take up to {api.W4_MAX_TOKENS} tokens, not {T}")
            self.y = torch.empty(T, H, dtype=torch.bfloat16, device=d)
            self.dev_status = torch.zeros(2, dtype=torch.int32, device=d)
            self.workspace = torch.empty(api.experts_w4_workspace_size(T, K, H, I),
                                         dtype=torch.uint8, device=d)
        else:
            if not fp4:
                self.hq = torch.empty(T, H, dtype=torch.uint8, device=d)
                self.hs = torch.empty(T, H // 128, dtype=torch.float32, device=d)
            self.lane = api.MoeLayerBuffers(T, E, K, H, I, T if capacity is None else capacity, d,
                                            packed=True, fp4=fp4, fp4_gscales=fp4_gscales)
            self.y, self.dev_status = self.lane.y, self.lane.dev_status

    def forward(self, x, residual, w13, w13_scale, w2, w2_scale, *, stream=None):
        """``x [T, H]`` bf16 (the sublayer before) joins ``residual [T, H]``
        (bf16 or fp32, updated in place).  Returns the routed branch's ``y
        [T, H]`` bf16, the block's own buffer; ``dev_status`` as of the calls,
        and ``router_status``, which keeps a timeout of the projection until
        the caller clears it."""
        api.moe_add_rms_norm(x, self.norm_weight, self.eps, residual=residual,
                             residual_out=residual, y=self.h, yq=self.hq, ys=self.hs,
                             stream=stream)
        api.moe_router_logits(self.h, self.router_weight, logits=self.logits,
                              dev_status=self.router_status, stream=stream)
        api.moe_router_topk(self.logits, self.K, topk_idx=self.topk_idx, topk_w=self.topk_w,
                            stream=stream, **self.router)
        if self.w4:
            return api.moe_experts_w4(self.h, self.topk_idx, self.topk_w, w13, w13_scale, w2,
                                      w2_scale, y=self.y, dev_status=self.dev_status,
                                      workspace=self.workspace, stream=stream)
        if self.fp4:
            return self.lane.forward(self.h, self.topk_idx, self.topk_w, w13, w13_scale, w2, w2_scale,
                                     stream=stream)
        self.lane.dispatch_fp8(self.hq, self.hs, self.topk_idx, stream=stream)
        self.lane.gemms(w13, w13_scale, w2, w2_scale, stream=stream)
        self.lane.combine(self.topk_w, self.y, stream=stream)
        return self.y
