"""The norm in front of the layer: residual addition, RMS norm and e4m3 rows
in one launch (``moe_rms_norm_quant``).

    r = rms_norm_quant(x, weight, residual)       # r.codes, r.scale, r.residual
    out = layer.stage(r.codes, topk_idx, topk_w, x_scale=r.scale)
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib as L
from ._args import check, current_raw_stream, empty_rows, ptr

_TYPES = {torch.bfloat16: L.MOE_TYPE_BF16, torch.float32: L.MOE_TYPE_F32}
_BF16, _F32, _CODES = (torch.bfloat16,), (torch.float32,), (torch.uint8, torch.float8_e4m3fn)


class NormOutput(NamedTuple):
    codes: Optional[torch.Tensor]     # uint8 [T, H], e4m3
    scale: Optional[torch.Tensor]     # float32 [T, H/128]
    y: Optional[torch.Tensor]         # bfloat16 [T, H]
    residual: Optional[torch.Tensor]  # [T, H], x + residual in the residual's type


def rms_norm_quant(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, *,
                   eps: float = 1e-6, codes: bool = True, bf16: bool = False,
                   out: Optional[NormOutput] = None) -> NormOutput:
    """RMS norm of ``x + residual`` with e4m3 rows (``codes``), BF16 rows
    (``bf16``) or both, and the new residual.

    x: bfloat16 [T, H]; weight: [H], residual: [T, H], each bfloat16 or
    float32.  x and the residual may have a row stride.  ``out`` supplies the
    output tensors instead (those that are None are not written);
    ``out.residual`` may be ``residual``.
    """
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError("x must be a [T, H] device tensor")
    shape, dev = x.shape, x.device
    index = dev.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return rms_norm_quant(x, weight, residual, eps=eps, codes=codes, bf16=bf16, out=out)
    T, H = shape
    check(x, "x", shape, _BF16, dev, True)
    check(weight, "weight", (H,), _TYPES, dev)
    if residual is not None:
        check(residual, "residual", shape, _TYPES, dev, True)
    if out is None:
        q = s = y = ro = None
        if codes:
            q = empty_rows(T, H, torch.uint8, dev)
            s = empty_rows(T, H // 128, torch.float32, dev)
        if bf16:
            y = empty_rows(T, H, torch.bfloat16, dev)
        if residual is not None:
            ro = empty_rows(T, H, residual.dtype, dev)
        out = NormOutput(q, s, y, ro)
    else:
        q, s, y, ro = out
        if q is not None:
            check(q, "out.codes", shape, _CODES, dev)
        if s is not None:
            check(s, "out.scale", (T, H // 128), _F32, dev)
        if y is not None:
            check(y, "out.y", shape, _BF16, dev)
        if ro is not None:
            if residual is None:
                raise ValueError("out.residual without a residual")
            check(ro, "out.residual", shape, (residual.dtype,), dev, True)
    rtype = r = rs = ros = 0
    if residual is not None:
        rtype, r, rs = _TYPES[residual.dtype], residual.data_ptr(), residual.stride(0)
        if ro is not None:
            ros = ro.stride(0)
    L.moe_rms_norm_quant(H, eps, rtype, _TYPES[weight.dtype], x.data_ptr(), x.stride(0), r, rs, weight.data_ptr(), T,
                         ptr(q), ptr(s), ptr(y), ptr(ro), ros, current_raw_stream(index))
    return out
