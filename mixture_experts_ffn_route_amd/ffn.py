"""The gated feed-forward block in bfloat16 with its gradients: an expert, a
shared expert or a dense layer before its quantisation, and to train it.

    y = gated_ffn(x, w13, w2)     # bfloat16 [T, H], differentiable
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable
from torch.autograd.graph import get_gradient_edge

from . import _lib as L
from ._args import check, current_raw_stream, empty_rows, ptr
from .linear import _workspace

_BF16, _F32 = (torch.bfloat16,), (torch.float32,)
_GRADS = {torch.bfloat16: L.MOE_TYPE_BF16, torch.float32: L.MOE_TYPE_F32}


def _sizes(x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor):
    if x.dim() != 2 or w2.dim() != 2 or not x.is_cuda:
        raise ValueError("x must be a [T, H] and w2 an [H, I] device tensor")
    T, H = x.shape
    I = w2.shape[1]
    check(x, "x", (T, H), _BF16, x.device, True)
    check(w13, "w13", (2 * I, H), _BF16, x.device)
    check(w2, "w2", (H, I), _BF16, x.device)
    return T, H, I


def _forward(x, w13, w2, out, gate_up: bool):
    """moe_ffn_forward of checked tensors on the current device."""
    (T, H), I, dev = x.shape, w2.shape[1], x.device
    if out is None:
        out = empty_rows(T, H, torch.bfloat16, dev)
    gu = empty_rows(T, 2 * I, torch.float32, dev) if gate_up else None
    h = empty_rows(T, I, torch.bfloat16, dev)
    ws_bytes = L.moe_ffn_workspace_query(T, H, I)[0]
    ws = _workspace(ws_bytes, dev)
    L.moe_ffn_forward(x.data_ptr(), x.stride(0), w13.data_ptr(), w2.data_ptr(), T, H, I, ptr(gu), h.data_ptr(),
                      out.data_ptr(), out.stride(0), ptr(ws), ws_bytes, current_raw_stream(dev.index))
    return out, gu, h


def _backward(dy, x, w13, w2, gu, h, dx, dw13, dw2, dw_type: int, accumulate: int) -> None:
    """moe_ffn_backward of checked tensors on the current device."""
    (T, H), I, dev = x.shape, w2.shape[1], x.device
    ws_bytes = 0 if dx is None and dw13 is None else L.moe_ffn_workspace_query(T, H, I)[1]
    ws = _workspace(ws_bytes, dev)
    L.moe_ffn_backward(dy.data_ptr(), dy.stride(0), x.data_ptr(), x.stride(0), w13.data_ptr(), w2.data_ptr(), ptr(gu),
                       ptr(h), T, H, I, ptr(dx), 0 if dx is None else dx.stride(0), ptr(dw13), ptr(dw2), dw_type,
                       accumulate, ptr(ws), ws_bytes, current_raw_stream(dev.index))


def gated_ffn_forward(x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, *, gate_up: bool = True,
                      out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor], torch.Tensor]:
    """``(silu(x Wg^T) * (x Wu^T)) w2^T`` without autograd (moe_ffn_forward):
    the output, and what gated_ffn_backward takes, the gate and up projections
    (``gate_up``: float32 [T, 2 I], else None) and h (bfloat16 [T, I])."""
    if x.is_cuda and x.device.index != torch.cuda.current_device():
        with torch.cuda.device(x.device):
            return gated_ffn_forward(x, w13, w2, gate_up=gate_up, out=out)
    T, H, I = _sizes(x, w13, w2)
    if out is not None:
        check(out, "out", (T, H), _BF16, x.device, True)
    return _forward(x, w13, w2, out, gate_up)


def gated_ffn_backward(dy: torch.Tensor, x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor,
                       gate_up: Optional[torch.Tensor], h: Optional[torch.Tensor], *, dx: Optional[torch.Tensor] = None,
                       dw13: Optional[torch.Tensor] = None, dw2: Optional[torch.Tensor] = None,
                       accumulate: bool = False) -> None:
    """Gradients of gated_ffn_forward's output (moe_ffn_backward) into those of
    ``dx`` (bfloat16 [T, H]), ``dw13`` and ``dw2`` (the weights' shapes, both
    bfloat16 or both float32) that are given.  ``accumulate``: the float32
    weight gradients are added to what is there.  ``gate_up`` may be None for
    dw2 alone, ``h`` without dw2."""
    if x.is_cuda and x.device.index != torch.cuda.current_device():
        with torch.cuda.device(x.device):
            return gated_ffn_backward(dy, x, w13, w2, gate_up, h, dx=dx, dw13=dw13, dw2=dw2, accumulate=accumulate)
    T, H, I = _sizes(x, w13, w2)
    dev = x.device
    check(dy, "dy", (T, H), _BF16, dev, True)
    if gate_up is not None:
        check(gate_up, "gate_up", (T, 2 * I), _F32, dev)
    elif dx is not None or dw13 is not None:
        raise ValueError("dx and dw13 need gate_up")
    if h is not None:
        check(h, "h", (T, I), _BF16, dev)
    elif dw2 is not None:
        raise ValueError("dw2 needs h")
    if dx is not None:
        check(dx, "dx", (T, H), _BF16, dev, True)
    kinds = {t.dtype for t in (dw13, dw2) if t is not None}
    if len(kinds) > 1:
        raise ValueError("dw13 and dw2 must have one type")
    if dw13 is not None:
        check(dw13, "dw13", (2 * I, H), _GRADS, dev)
    if dw2 is not None:
        check(dw2, "dw2", (H, I), _GRADS, dev)
    _backward(dy, x, w13, w2, gate_up, h, dx, dw13, dw2, _GRADS[kinds.pop()] if kinds else L.MOE_TYPE_BF16,
              int(accumulate))


_MAX_STRIDE = 1 << 20  # of rows that the kernels read, in values


def _readable_rows(dy: torch.Tensor) -> torch.Tensor:
    """dy, or a copy of one that is broadcast or a view that the kernels do not
    read."""
    T, H = dy.shape
    row = dy.stride(0)
    if dy.stride(1) != 1 or dy.data_ptr() % 16 or (T > 1 and (row < H or row % 8 or row > _MAX_STRIDE)):
        return dy.clone(memory_format=torch.contiguous_format)
    return dy


# Mark on a leaf's gradient node: an eager graph of the default stream holds it.
_EAGER = "moe_gated_ffn_eager"


class _GatedFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w13, w2):
        need_x, need_w13, need_w2 = ctx.needs_input_grad
        out, gu, h = _forward(x, w13, w2, None, need_x or need_w13)
        ctx.save_for_backward(x, w13, w2, gu, h if need_w2 else None)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w13, w2, gu, h = ctx.saved_tensors
        need_x, need_w13, need_w2 = ctx.needs_input_grad
        T, H = x.shape
        dy = _readable_rows(dy)
        dx = empty_rows(T, H, torch.bfloat16, x.device) if need_x else None
        dw13 = empty_rows(w13.shape[0], H, torch.bfloat16, x.device) if need_w13 else None
        dw2 = empty_rows(H, w2.shape[1], torch.bfloat16, x.device) if need_w2 else None
        if x.device.index != torch.cuda.current_device():
            with torch.cuda.device(x.device):
                _backward(dy, x, w13, w2, gu, h, dx, dw13, dw2, L.MOE_TYPE_BF16, 0)
        else:
            _backward(dy, x, w13, w2, gu, h, dx, dw13, dw2, L.MOE_TYPE_BF16, 0)
        return dx, dw13, dw2


def gated_ffn(x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor) -> torch.Tensor:
    """``(silu(x Wg^T) * (x Wu^T)) w2^T`` in bfloat16 [T, H], differentiable in
    x, w13 and w2.

    x: bfloat16 [T, H], the rows may have a stride; w13: bfloat16 [2 I, H], gate
    rows Wg and then up rows Wu; w2: bfloat16 [H, I].  H and I are multiples of
    8.  Gradients are bfloat16; gated_ffn_backward also gives and accumulates
    float32 weight gradients.  As with any backward pass, a capture into a graph
    must not meet leaves of an eager graph that is still alive; that is refused
    where this function made the eager graph.  Derivatives are those of reverse
    mode: a tangent of forward mode on an input is refused."""
    # The level by itself first: unpack_dual takes 0.5 us a tensor.
    if forward_ad._current_level >= 0 and any(forward_ad.unpack_dual(t).tangent is not None for t in (x, w13, w2)):
        raise NotImplementedError("gated_ffn has no forward-mode derivative")
    if not (torch.is_grad_enabled() and (x.requires_grad or w13.requires_grad or w2.requires_grad)):
        return gated_ffn_forward(x, w13, w2, gate_up=False)[0]
    if x.is_cuda and x.device.index != torch.cuda.current_device():
        with torch.cuda.device(x.device):
            return gated_ffn(x, w13, w2)
    _sizes(x, w13, w2)
    if torch.cuda.is_current_stream_capturing():
        # The captured backward would make the default stream, on which an eager
        # graph's nodes were born, wait within the capture; it cannot be part of
        # one, and the process ends.
        for t in (x, w13, w2):
            if t.requires_grad and t.is_leaf and _EAGER in get_gradient_edge(t).node.metadata:
                raise RuntimeError("gated_ffn is being captured while an eager graph of one of its leaves lives: "
                                   "release that graph first, or capture gated_ffn_forward and gated_ffn_backward")
        return _GatedFFN.apply(x, w13, w2)
    y = _GatedFFN.apply(x, w13, w2)
    if current_raw_stream(x.device.index) == 0:
        for node, _ in y.grad_fn.next_functions:
            if node is not None and node.name() == "torch::autograd::AccumulateGrad":
                node.metadata[_EAGER] = True
    return y
