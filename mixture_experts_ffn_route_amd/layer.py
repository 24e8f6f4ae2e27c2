"""A small owner of one layer handle: torch provides the device memory and
the stream, the HIP library does every step of the forward.

    layer = MoELayer(cfg, w13, w13_scale, w2, w2_scale, expected_m=..., max_rows=...)
    out = layer.stage(x, topk_idx, topk_w)      # x: bf16 [T, H] (or e4m3 codes + x_scale)
    layer.forward()                             # writes `out` on the current stream
"""

from __future__ import annotations

from typing import Optional

import torch

from . import _lib as L
from ._args import check, current_raw_stream, empty_rows, ptr

_BF16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)
_CODES = (torch.uint8, torch.float8_e4m3fn)


class MoELayer:
    def __init__(self, hidden: int, intermediate: int, num_experts: int, top_k: int,
                 w13: torch.Tensor, w13_scale: torch.Tensor, w2: torch.Tensor, w2_scale: torch.Tensor, *,
                 expected_m: int, max_rows: int, capacity_factor: float = 1.0,
                 weight_format: int = L.MOE_WEIGHT_E4M3_BLOCK128, act_format: int = L.MOE_ACT_E4M3_1X128,
                 flags: int = L.MOE_FLAG_CHECK_ROUTES, workspace: Optional[torch.Tensor] = None):
        for t in (w13, w13_scale, w2, w2_scale):
            if not (t.is_cuda and t.is_contiguous()):
                raise ValueError("weights must be contiguous device tensors")
        self.cfg = L.make_config(hidden, intermediate, num_experts, top_k, weight_format, act_format, flags)
        self.hidden, self.top_k = hidden, top_k
        self.max_rows, self.capacity_factor = max_rows, capacity_factor
        self.ws_bytes = L.moe_workspace_query(self.cfg, expected_m, max_rows, capacity_factor)
        if workspace is None:
            workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=w13.device)
        elif workspace.numel() < self.ws_bytes or not workspace.is_contiguous():
            raise ValueError("workspace too small, or not contiguous")
        self.workspace = workspace
        self._keep = (w13, w13_scale, w2, w2_scale)  # the handle reads these in place
        with torch.cuda.device(workspace.device):
            self.handle = L.moe_layer_create(self.cfg, expected_m, max_rows, capacity_factor, ptr(w13),
                                             ptr(w13_scale), ptr(w2), ptr(w2_scale), ptr(workspace),
                                             self.ws_bytes, self._stream())
        self._staged = None

    @staticmethod
    def _stream() -> int:
        return torch.cuda.current_stream().cuda_stream

    def _elsewhere(self) -> bool:
        """Whether another device than the layer's is current; its calls then
        switch to it, for launches go to the current device's stream."""
        return self.workspace.device.index != torch.cuda.current_device()

    def stage(self, x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
              x_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        if self._elsewhere():
            with torch.cuda.device(self.workspace.device):
                return self.stage(x, topk_idx, topk_w, x_scale, out)
        T = x.shape[0]
        if out is None:
            out = torch.empty((T, self.hidden), dtype=torch.bfloat16, device=x.device)
        for t in (x, topk_idx, topk_w, out) + ((x_scale,) if x_scale is not None else ()):
            if not t.is_contiguous():
                raise ValueError("inputs must be contiguous")
        L.moe_stage_inputs(self.handle, ptr(x), ptr(x_scale), ptr(topk_idx), ptr(topk_w), T, ptr(out),
                           self._stream())
        self._staged = (x, topk_idx, topk_w, x_scale, out)  # keep alive until forward
        return out

    def forward(self) -> None:
        if self._elsewhere():
            with torch.cuda.device(self.workspace.device):
                return self.forward()
        L.moe_layer_forward(self.handle, self._stream())

    def forward_noalloc(self, x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor, out: torch.Tensor,
                        x_scale: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None) -> None:
        """Stage + forward with the per-call regions in the library's static
        device scratch (moe_layer_forward_noalloc): ``out`` and the optional
        int32 ``status`` word are caller tensors, nothing is allocated."""
        if self._elsewhere():
            with torch.cuda.device(self.workspace.device):
                return self.forward_noalloc(x, topk_idx, topk_w, out, x_scale, status)
        for t in (x, topk_idx, topk_w, out) + tuple(t for t in (x_scale, status) if t is not None):
            if not t.is_contiguous():
                raise ValueError("inputs must be contiguous")
        L.moe_layer_forward_noalloc(self.handle, ptr(x), ptr(x_scale), ptr(topk_idx), ptr(topk_w), x.shape[0],
                                    ptr(out), ptr(status), self._stream())

    def decode(self, x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
               x_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The whole layer for at most 16 tokens in two launches
        (moe_layer_decode): x bfloat16 [T, H], or e4m3 codes with x_scale.
        Faster than stage + forward up to about 48 routes to this layer's
        experts (FP8 weights; 16 and 8 with rows longer than 7168 and 10240) or
        40 and 12 tokens (MXFP8); from there to 16 tokens with all routes up to
        12 and 22 % slower, with the longer rows up to 40.
        The optional int32 ``status`` word receives the call's MOE_DEV_*
        bits."""
        dev = self.workspace.device
        if self._elsewhere():
            with torch.cuda.device(dev):
                return self.decode(x, topk_idx, topk_w, x_scale, out, status)
        T = x.shape[0]
        shape, routes = (T, self.hidden), (T, self.top_k)
        check(x, "x", shape, _BF16 if x_scale is None else _CODES, dev)
        if x_scale is not None:
            check(x_scale, "x_scale", (T, self.hidden // 128), _F32, dev)
        check(topk_idx, "topk_idx", routes, _I32, dev)
        check(topk_w, "topk_w", routes, _F32, dev)
        if out is None:
            out = empty_rows(T, self.hidden, torch.bfloat16, dev)
        else:
            check(out, "out", shape, _BF16, dev)
        if status is not None:
            check(status, "status", (1,), _I32, dev)
        L.moe_layer_decode(self.handle, x.data_ptr(), ptr(x_scale), topk_idx.data_ptr(), topk_w.data_ptr(), T,
                           out.data_ptr(), ptr(status), current_raw_stream(dev.index))
        return out

    def status(self) -> int:
        if self._elsewhere():
            with torch.cuda.device(self.workspace.device):
                return self.status()
        return L.moe_read_status(self.handle, self._stream())

    def region(self, name: str, dtype: torch.dtype, shape=None) -> torch.Tensor:
        """A device view of a workspace region (no copy)."""
        address, nbytes = L.moe_layer_region(self.handle, L.REGIONS[name])
        off = address - self.workspace.data_ptr()
        view = self.workspace[off:off + nbytes].view(dtype)
        return view if shape is None else view[: int(torch.tensor(shape).prod())].view(*shape)

    def tactic(self) -> dict:
        return L.moe_layer_tactic(self.handle)

    def profile(self, enable=True, kernels=None) -> None:
        """Time every kernel class (``enable`` true), the named ``kernels``
        only (e.g. ``("fc1",)``), or stop (``enable`` false)."""
        mask = 0
        if enable:
            mask = L.PROFILE_ALL if kernels is None else sum(1 << L.KERNELS.index(k) for k in kernels)
        L.moe_profile_enable(self.handle, mask)

    def profile_read(self) -> dict:
        return L.moe_profile_read(self.handle)

    def close(self) -> None:
        if getattr(self, "handle", None):
            L.moe_layer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
