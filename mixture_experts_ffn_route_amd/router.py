"""The router in front of the layer: a small owner of one router handle.

    router = MoERouter(gate_weight, top_k=8, max_rows=4096, score="sigmoid", bias=bias, num_groups=8, top_groups=4)
    topk_idx, topk_w = router.route(x)            # x: bf16 [T, H]
    out = layer.stage(x, topk_idx, topk_w)
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _lib as L
from ._args import check, current_raw_stream, empty_rows, ptr

_SCORES = {"softmax": L.MOE_SCORE_SOFTMAX, "sigmoid": L.MOE_SCORE_SIGMOID}
_BF16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)


class MoERouter:
    """``weight``: bfloat16 [E, H], the gate of the whole model; ``bias``:
    float32 [E], added to sigmoid scores for the selection.  The experts
    [expert_base, expert_base + local_experts) are this GPU's (all of them by
    default); routes to others come out as -1.  The weight is read in place
    while the router exists, the bias is copied; one router's calls must not
    overlap on the device, nor with its creation (on the stream current then)."""

    def __init__(self, weight: torch.Tensor, top_k: int, *, max_rows: int, score: str = "softmax",
                 bias: Optional[torch.Tensor] = None, num_groups: int = 1, top_groups: int = 1,
                 renormalize: bool = True, scale: float = 1.0, expert_base: int = 0,
                 local_experts: Optional[int] = None, workspace: Optional[torch.Tensor] = None):
        if weight.dim() != 2 or not weight.is_cuda:
            raise ValueError("weight must be an [E, H] device tensor")
        if score not in _SCORES:
            raise ValueError(f"score must be one of {tuple(_SCORES)}")
        E, H = weight.shape
        self.device = weight.device
        check(weight, "weight", (E, H), _BF16, self.device)
        if bias is not None:
            check(bias, "bias", (E,), _F32, self.device)
        if local_experts is None:
            local_experts = E - expert_base
        self.cfg = L.moe_router_config_t(H, E, top_k, _SCORES[score], num_groups, top_groups, int(renormalize), scale,
                                         expert_base, local_experts)
        self.hidden, self.top_k, self.max_rows = H, top_k, max_rows
        self.ws_bytes = L.moe_router_workspace_query(self.cfg, max_rows)
        if workspace is None:
            workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        elif (workspace.numel() * workspace.element_size() < self.ws_bytes or workspace.device != self.device
              or not workspace.is_contiguous()):
            raise ValueError("workspace too small, on another device, or not contiguous")
        self.workspace = workspace
        self._keep = (weight, bias)  # the handle reads the weight in place; the bias until its copy is made
        with torch.cuda.device(self.device):
            self.handle = L.moe_router_create(self.cfg, max_rows, ptr(weight), ptr(bias), ptr(workspace),
                                              self.ws_bytes, current_raw_stream(self.device.index))

    def route(self, x: torch.Tensor, topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
              ids: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Experts and weights of the rows ``x`` (bfloat16 [T, H], T at most
        max_rows; the rows may have a stride), as the layer takes them.
        ``ids`` receives the experts' numbers in the whole model."""
        dev = self.device
        if dev.index != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return self.route(x, topk_idx, topk_w, ids)
        T = x.shape[0]
        check(x, "x", (T, self.hidden), _BF16, dev, True)
        shape = (T, self.top_k)
        if topk_idx is None:
            topk_idx = empty_rows(T, self.top_k, torch.int32, dev)
        else:
            check(topk_idx, "topk_idx", shape, _I32, dev)
        if topk_w is None:
            topk_w = empty_rows(T, self.top_k, torch.float32, dev)
        else:
            check(topk_w, "topk_w", shape, _F32, dev)
        if ids is not None:
            check(ids, "ids", shape, _I32, dev)
        L.moe_router_forward(self.handle, x.data_ptr(), x.stride(0), T, topk_idx.data_ptr(), topk_w.data_ptr(),
                             ptr(ids), current_raw_stream(dev.index))
        return topk_idx, topk_w

    def close(self) -> None:
        if getattr(self, "handle", None):
            L.moe_router_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
