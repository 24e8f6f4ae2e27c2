"""The gated feed-forward block in bfloat16 with its gradients: an expert, a
shared expert or a dense layer before its quantisation, and to train it.

    y = gated_ffn(x, w13, w2)     # bfloat16 [T, H], differentiable
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch
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


def gated_ffn_forward(x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, *, gate_up: bool = True,
                      out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor], torch.Tensor]:
    """``(silu(x Wg^T) * (x Wu^T)) w2^T`` without autograd (moe_ffn_forward):
    the output, and what gated_ffn_backward takes, the gate and up projections
    (``gate_up``: float32 [T, 2 I], else None) and h (bfloat16 [T, I])."""
    if x.is_cuda and x.device.index != torch.cuda.current_device():
        with torch.cuda.device(x.device):
            return gated_ffn_forward(x, w13, w2, gate_up=gate_up, out=out)
    T, H, I = _sizes(x, w13, w2)
    dev = x.device
    if out is None:
        out = empty_rows(T, H, torch.bfloat16, dev)
    else:
        check(out, "out", (T, H), _BF16, dev, True)
    gu = empty_rows(T, 2 * I, torch.float32, dev) if gate_up else None
    h = empty_rows(T, I, torch.bfloat16, dev)
    ws_bytes = L.moe_ffn_workspace_query(T, H, I)[0]
    ws = _workspace(ws_bytes, dev)
    L.moe_ffn_forward(x.data_ptr(), x.stride(0), w13.data_ptr(), w2.data_ptr(), T, H, I, ptr(gu), h.data_ptr(),
                      out.data_ptr(), out.stride(0), ptr(ws), ws_bytes, current_raw_stream(dev.index))
    return out, gu, h


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
    ws_bytes = L.moe_ffn_workspace_query(T, H, I)[1]
    ws = _workspace(ws_bytes, dev)
    L.moe_ffn_backward(dy.data_ptr(), dy.stride(0), x.data_ptr(), x.stride(0), w13.data_ptr(), w2.data_ptr(),
                       ptr(gate_up), ptr(h), T, H, I, ptr(dx), 0 if dx is None else dx.stride(0), ptr(dw13), ptr(dw2),
                       _GRADS[kinds.pop()] if kinds else L.MOE_TYPE_BF16, int(accumulate), ptr(ws), ws_bytes,
                       current_raw_stream(dev.index))


class _GatedFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w13, w2):
        need_x, need_w13, need_w2 = ctx.needs_input_grad
        out, gu, h = gated_ffn_forward(x, w13, w2, gate_up=need_x or need_w13)
        ctx.save_for_backward(x, w13, w2, gu, h if need_w2 else None)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w13, w2, gu, h = ctx.saved_tensors
        need_x, need_w13, need_w2 = ctx.needs_input_grad
        if dy.stride(-1) != 1 or (dy.shape[0] > 1 and (dy.stride(0) < dy.shape[1] or dy.stride(0) % 8)) or \
                dy.data_ptr() % 16:
            dy = dy.clone(memory_format=torch.contiguous_format)  # broadcast, or a view that the kernels do not read
        dx = empty_rows(*x.shape, torch.bfloat16, x.device) if need_x else None
        dw13 = torch.empty_like(w13) if need_w13 else None
        dw2 = torch.empty_like(w2) if need_w2 else None
        gated_ffn_backward(dy, x, w13, w2, gu, h, dx=dx, dw13=dw13, dw2=dw2)
        return dx, dw13, dw2


_BORN = "moe_gated_ffn_stream"  # mark on a leaf's gradient node: the stream of the graph that it was met in


def _leaf_nodes(leaves, dev) -> list:
    """The leaves' gradient nodes, marked; to be held until the new graph holds
    them.  Refuses a capture with leaves whose gradient nodes an eager graph of the
    default stream keeps alive: the captured backward would make that stream wait
    within the capture, which it cannot be part of, and ends the process."""
    stream = current_raw_stream(dev.index)
    capturing = torch.cuda.is_current_stream_capturing()
    nodes = []
    for t in leaves:
        if t.requires_grad and t.is_leaf:
            nodes.append(get_gradient_edge(t).node)
            if nodes[-1].metadata.setdefault(_BORN, stream) == 0 and capturing:
                raise RuntimeError("gated_ffn is being captured while an eager graph of one of its leaves lives: "
                                   "release that graph first, or capture gated_ffn_forward and gated_ffn_backward")
    return nodes


def gated_ffn(x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor) -> torch.Tensor:
    """``(silu(x Wg^T) * (x Wu^T)) w2^T`` in bfloat16 [T, H], differentiable in
    x, w13 and w2.

    x: bfloat16 [T, H], the rows may have a stride; w13: bfloat16 [2 I, H], gate
    rows Wg and then up rows Wu; w2: bfloat16 [H, I].  H and I are multiples of
    8.  Gradients are bfloat16; gated_ffn_backward also gives and accumulates
    float32 weight gradients.  As with any backward pass, a capture into a graph
    must not meet leaves of an eager graph that is still alive; that is refused
    where this function made the eager graph."""
    if torch.is_grad_enabled() and (x.requires_grad or w13.requires_grad or w2.requires_grad):
        nodes = _leaf_nodes((x, w13, w2), x.device) if x.is_cuda else None  # noqa: F841 (held over the call)
        return _GatedFFN.apply(x, w13, w2)
    return gated_ffn_forward(x, w13, w2, gate_up=False)[0]
