"""The dense FP8 products beside the experts: e4m3 rows times e4m3 weights with
one scale per block of 128, and the shared expert made of two of them.

    r = rms_norm_quant(x, norm_weight, residual)
    q = fp8_matmul(r.codes, r.scale, w, w_scale)             # bfloat16 [T, N]
    shared = MoESharedExpert(w13, w13_scale, w2, w2_scale)
    out = shared.forward(r.codes, r.scale, add=routed)       # bfloat16 [T, H]
"""

from __future__ import annotations

from typing import Optional

import torch

from . import _lib as L
from ._args import check, current_raw_stream, empty_rows, ptr

_BF16, _F32 = (torch.bfloat16,), (torch.float32,)
_CODES = (torch.uint8, torch.float8_e4m3fn)


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _workspace(nbytes: int, dev):
    """A call's own workspace (the allocator keeps it for this stream until the
    call's launches are done), or None."""
    return torch.empty_strided((nbytes,), (1,), dtype=torch.uint8, device=dev) if nbytes else None


def _rows_out(T: int, N: int, add, out, dev):
    """Checks ``add`` and ``out`` ([T, N]); returns out, made if it is None,
    and add's row stride."""
    if add is not None:
        check(add, "add", (T, N), _BF16, dev, True)
    if out is None:
        out = empty_rows(T, N, torch.bfloat16, dev)
    else:
        check(out, "out", (T, N), _BF16, dev, True)
    return out, 0 if add is None else add.stride(0)


def fp8_matmul(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, *,
               add: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``x w^T`` (``+ add``) in bfloat16 [M, N] (moe_fp8_matmul).

    x: e4m3 codes [M, K] (uint8 or float8_e4m3fn) with x_scale, float32
    [M, ceil(K/128)]; w: codes [N, K] with w_scale, float32 [ceil(N/128),
    ceil(K/128)].  K is a multiple of 16.  x, w, add and out may have a row
    stride; out may be add.  For serving: no derivative, add's either."""
    if x.dim() != 2 or w.dim() != 2 or not x.is_cuda:
        raise ValueError("x and w must be 2-D device tensors")
    dev = x.device
    index = dev.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return fp8_matmul(x, x_scale, w, w_scale, add=add, out=out)
    M, K = x.shape
    N = w.shape[0]
    check(x, "x", (M, K), _CODES, dev, True)
    check(x_scale, "x_scale", (M, _blocks(K)), _F32, dev)
    check(w, "w", (N, K), _CODES, dev, True)
    check(w_scale, "w_scale", (_blocks(N), _blocks(K)), _F32, dev)
    out, add_stride = _rows_out(M, N, add, out, dev)
    ws_bytes = L.moe_fp8_matmul_workspace_query(M, N, K)
    ws = _workspace(ws_bytes, dev)
    L.moe_fp8_matmul(x.data_ptr(), x.stride(0), x_scale.data_ptr(), w.data_ptr(), w.stride(0), w_scale.data_ptr(), M,
                     N, K, ptr(add), add_stride, out.data_ptr(), out.stride(0), ptr(ws), ws_bytes,
                     current_raw_stream(index))
    return out


class MoESharedExpert:
    """The expert that every token takes: ``w13`` e4m3 [2 I, H] (gate rows, then
    up rows) and ``w2`` [H, I] with float32 scales per 128 x 128 block.  The
    weights are read in place; calls share nothing, so they may overlap."""

    def __init__(self, w13: torch.Tensor, w13_scale: torch.Tensor, w2: torch.Tensor, w2_scale: torch.Tensor):
        if w2.dim() != 2 or not w2.is_cuda:
            raise ValueError("w2 must be an [H, I] device tensor")
        H, I = w2.shape
        dev = w2.device
        check(w13, "w13", (2 * I, H), _CODES, dev)
        check(w13_scale, "w13_scale", (_blocks(2 * I), _blocks(H)), _F32, dev)
        check(w2, "w2", (H, I), _CODES, dev)
        check(w2_scale, "w2_scale", (_blocks(H), _blocks(I)), _F32, dev)
        L.moe_ffn_fp8_workspace_query(1, H, I)  # refuses what the kernels do not take
        self.hidden, self.intermediate, self.device = H, I, dev
        self.w13, self.w13_scale, self.w2, self.w2_scale = w13, w13_scale, w2, w2_scale

    def forward(self, x: torch.Tensor, x_scale: torch.Tensor, add: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x: e4m3 codes [T, H] with x_scale, float32 [T, H/128], as
        rms_norm_quant gives them.  Returns the expert's output (``+ add``) in
        bfloat16 [T, H]; x, add and out may have a row stride, out may be
        add.  For serving: no derivative, add's either."""
        dev, H = self.device, self.hidden
        index = dev.index
        if index != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return self.forward(x, x_scale, add, out)
        T = x.shape[0]
        check(x, "x", (T, H), _CODES, dev, True)
        check(x_scale, "x_scale", (T, H // 128), _F32, dev)
        out, add_stride = _rows_out(T, H, add, out, dev)
        ws_bytes = L.moe_ffn_fp8_workspace_query(T, H, self.intermediate)
        ws = _workspace(ws_bytes, dev)
        L.moe_ffn_fp8(x.data_ptr(), x.stride(0), x_scale.data_ptr(), self.w13.data_ptr(), self.w13_scale.data_ptr(),
                      self.w2.data_ptr(), self.w2_scale.data_ptr(), T, H, self.intermediate, ptr(add), add_stride,
                      out.data_ptr(), out.stride(0), ptr(ws), ws_bytes, current_raw_stream(index))
        return out
