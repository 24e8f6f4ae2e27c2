"""The norm in front of the layer: residual addition, RMS norm and e4m3 rows
in one launch (``moe_rms_norm_quant``).

    r = rms_norm_quant(x, weight, residual)       # r.codes, r.scale, r.residual
    out = layer.stage(r.codes, topk_idx, topk_w, x_scale=r.scale)
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib as L

_TYPES = {torch.bfloat16: L.MOE_TYPE_BF16, torch.float32: L.MOE_TYPE_F32}


class NormOutput(NamedTuple):
    codes: Optional[torch.Tensor]     # uint8 [T, H], e4m3
    scale: Optional[torch.Tensor]     # float32 [T, H/128]
    y: Optional[torch.Tensor]         # bfloat16 [T, H]
    residual: Optional[torch.Tensor]  # [T, H], x + residual in the residual's type


def _rows(t: torch.Tensor, name: str, shape, dtypes, device, strided: bool = False) -> torch.Tensor:
    if t.shape != shape or t.dtype not in dtypes or t.device != device:
        raise ValueError(f"{name} must be {tuple(shape)} of {dtypes} on {device}, got {tuple(t.shape)} {t.dtype} on "
                         f"{t.device}")
    if not (t.is_contiguous() or (strided and t.stride(-1) == 1)):
        raise ValueError(f"{name} must be contiguous" + (" along its last dimension" if strided else ""))
    return t


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
    T, H = x.shape
    dev = x.device
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return rms_norm_quant(x, weight, residual, eps=eps, codes=codes, bf16=bf16, out=out)
    _rows(x, "x", x.shape, (torch.bfloat16,), dev, True)
    _rows(weight, "weight", (H,), _TYPES, dev)
    if residual is not None:
        _rows(residual, "residual", x.shape, _TYPES, dev, True)
    if out is None:
        empty = torch.empty
        out = NormOutput(empty((T, H), dtype=torch.uint8, device=dev) if codes else None,
                         empty((T, H // 128), dtype=torch.float32, device=dev) if codes else None,
                         empty((T, H), dtype=torch.bfloat16, device=dev) if bf16 else None,
                         None if residual is None else empty((T, H), dtype=residual.dtype, device=dev))
    else:
        if out.codes is not None:
            _rows(out.codes, "out.codes", x.shape, (torch.uint8, torch.float8_e4m3fn), dev)
        if out.scale is not None:
            _rows(out.scale, "out.scale", (T, H // 128), (torch.float32,), dev)
        if out.y is not None:
            _rows(out.y, "out.y", x.shape, (torch.bfloat16,), dev)
        if out.residual is not None:
            if residual is None:
                raise ValueError("out.residual without a residual")
            _rows(out.residual, "out.residual", x.shape, (residual.dtype,), dev, True)
    r, ro = residual, out.residual
    ptr = torch.Tensor.data_ptr
    L.moe_rms_norm_quant(H, eps, _TYPES[r.dtype] if r is not None else 0, _TYPES[weight.dtype], ptr(x), x.stride(0),
                         0 if r is None else ptr(r), 0 if r is None else r.stride(0), ptr(weight), T,
                         0 if out.codes is None else ptr(out.codes), 0 if out.scale is None else ptr(out.scale),
                         0 if out.y is None else ptr(out.y), 0 if ro is None else ptr(ro),
                         0 if ro is None else ro.stride(0), torch.cuda.current_stream().cuda_stream)
    return out
