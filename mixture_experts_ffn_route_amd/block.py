"""The MoE block of a decoder layer: residual norm, router and layer.

    block = MoEBlock(norm_weight, router, layer)
    out, residual = block.forward(attention_out, residual)

``out`` is what the next layer adds to ``residual``.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _lib as L
from ._args import check
from .layer import MoELayer
from .norm import rms_norm_quant
from .router import MoERouter

# Batches of up to so many tokens, expected to have so many routes here (tokens
# top_k local_experts / num_experts), take the few-token layer, which is faster
# than stage + forward up to there.  us, few-token / stage + forward:
#   all experts here   FP8 H=7168 I=2048 K=8    T=1 66/84, 6 195/201, 8 212/206
#                      FP8 H=2048 I=768 K=6     T=1 18/34, 8 38/40, 10 43/41
#                      MXFP8, the first sizes   T=1 68/88, 4 163/175, 6 201/201, 8 219/209
#                      MXFP8, the second        T=8 38/40, 10 42/40
#   an eighth of them  FP8, the first           T=1 15/34, 8 62/87, 16 94/105
#                      FP8, the second          T=16 24/35
#                      MXFP8, the first         T=8 60/87, 12 100/104, 16 124/116
#                      MXFP8, the second        T=16 25/35
# Longer FP8 rows keep more of the token operand in registers, or spill it (I=1536
# K=4 of 16, all here: H=10240 T=4 108/113, 8 140/126; H=12288 T=1 73/97, 4 145/126;
# H=16384 T=1 90/120, 4 183/157).
FEW_TOKENS, FEW_ROUTES = 16, 48
FEW_ROUTES_LONG = ((10240, 8), (7168, 16))   # (rows longer than, routes)
FEW_TOKENS_MX, FEW_ROUTES_MX = 12, 40


class MoEBlock:
    """``router`` has to give local expert ids of ``layer`` (its
    local_experts are the layer's).  FP8 layers take the norm's e4m3 rows,
    MXFP8 layers its BF16 rows, which the router reads in both cases."""

    def __init__(self, norm_weight: torch.Tensor, router: MoERouter, layer: MoELayer, *, eps: float = 1e-6):
        if router.hidden != layer.hidden or router.top_k != layer.top_k:
            raise ValueError(f"router (hidden {router.hidden}, top_k {router.top_k}) and layer (hidden "
                             f"{layer.hidden}, top_k {layer.top_k}) do not fit")
        if router.cfg.local_experts != layer.cfg.num_experts:
            raise ValueError(f"the router maps to {router.cfg.local_experts} local experts, the layer has "
                             f"{layer.cfg.num_experts}")
        if router.device != layer.workspace.device:
            raise ValueError(f"router on device {router.device}, layer on {layer.workspace.device}")
        self.norm_weight, self.router, self.layer, self.eps = norm_weight, router, layer, eps
        self.fp8 = layer.cfg.act_format == L.MOE_ACT_E4M3_1X128
        tokens, routes = FEW_TOKENS_MX, FEW_ROUTES_MX
        if self.fp8:
            tokens = FEW_TOKENS
            routes = next((r for hidden, r in FEW_ROUTES_LONG if layer.hidden > hidden), FEW_ROUTES)
        self.few = min(tokens, routes * router.cfg.num_experts // (router.top_k * router.cfg.local_experts))
        if layer.capacity_factor < 1.0:
            self.few = 0  # the few-token layer drops no routes

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """x: bfloat16 [T, H]; residual: [T, H] or None.  Returns the experts'
        output (bfloat16 [T, H]) and x + residual.  The optional int32
        ``status`` word ([1]) receives the call's MOE_DEV_* bits
        (``layer.status()`` has those of stage + forward only)."""
        if status is not None:
            check(status, "status", (1,), (torch.int32,), self.router.device)
        n = rms_norm_quant(x, self.norm_weight, residual, eps=self.eps, codes=self.fp8, bf16=True)
        idx, w = self.router.route(n.y)
        rows, scale = (n.codes, n.scale) if self.fp8 else (n.y, None)
        if x.shape[0] <= self.few:
            out = self.layer.decode(rows, idx, w, x_scale=scale, out=out, status=status)
        else:
            out = self.layer.stage(rows, idx, w, x_scale=scale, out=out)
            self.layer.forward()
            if status is not None:
                status.copy_(self.layer.region("status", torch.int32)[:1])
        return out, n.residual
