"""Edges of the gated block's derivatives: what it cannot give is refused, which
gradients of the output it copies, what dw2 alone takes."""

import pytest
import torch
import torch.autograd.forward_ad as fwd

import mixture_experts_ffn_route_amd as m
from mixture_experts_ffn_route_amd import _lib as L
from mixture_experts_ffn_route_amd import ffn
from tests import dense_util as D

DEVICES = ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)]


@pytest.mark.parametrize("device", DEVICES)
@pytest.mark.parametrize("which", range(3))
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("enabled", [False, True])
def test_a_tangent_is_refused(device, which, grad, enabled):
    """On the CPU before the tensors' device is refused."""
    args = list(D.ffn_inputs(3, 16, 8, 0, device=device)[:3])
    args[(which + 1) % 3].requires_grad_(grad)
    with torch.set_grad_enabled(enabled), fwd.dual_level():
        args[which] = fwd.make_dual(args[which], torch.ones_like(args[which]))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            m.gated_ffn(*args)


@pytest.mark.gpu
def test_a_level_without_tangents_on_the_inputs():
    x, w13, w2, dy = D.ffn_inputs(3, 16, 8, 0)
    want = m.gated_ffn(x, w13, w2)
    x.requires_grad_(True)
    (grad,) = torch.autograd.grad(m.gated_ffn(x, w13, w2), (x,), dy)
    with fwd.dual_level():
        other = fwd.make_dual(dy, dy)
        assert torch.equal(m.gated_ffn(x.detach(), w13, w2), want)
        y = m.gated_ffn(x, w13, w2)
        assert fwd.unpack_dual(y).tangent is None and fwd.unpack_dual(other).tangent is not None
        (got,) = torch.autograd.grad(y, (x,), dy)
    assert torch.equal(got, grad)


def _views(device):
    """Gradients of [3, 16] as views, and whether the kernels read them in place."""
    def rows(stride, at=0):
        gen = torch.Generator(device=device).manual_seed(stride)
        flat = torch.randn(at + 2 * stride + 16, generator=gen, device=device).bfloat16()
        return flat.as_strided((3, 16), (stride, 1), at)

    return [(rows(16), True), (rows(24), True), (rows(1 << 20), True), (rows((1 << 20) + 8), False), (rows(1 << 21), False),
            (rows(20), False), (rows(8), False), (rows(24, 4), False), (rows(16)[:1].expand(3, 16), False),
            (rows(16).t().contiguous().t(), False)]


@pytest.mark.parametrize("k", range(10))
def test_which_gradients_are_copied(k):
    dy, in_place = _views("cpu")[k]
    if dy.data_ptr() % 16 and in_place:
        pytest.skip("the allocator gave no 16-byte alignment")
    got = ffn._readable_rows(dy)
    assert (got is dy) == in_place and (in_place or got.is_contiguous())


@pytest.mark.gpu
@pytest.mark.parametrize("k", range(10))
def test_backward_takes_any_view(k):
    """Among them a slice of columns of a buffer wider than the kernels' strides."""
    x, w13, w2, _ = D.ffn_inputs(3, 16, 8, 1)
    x.requires_grad_(True)
    dy, _ = _views("cuda")[k]
    (want,) = torch.autograd.grad(m.gated_ffn(x, w13, w2), (x,), dy.clone(memory_format=torch.contiguous_format))
    (got,) = torch.autograd.grad(m.gated_ffn(x, w13, w2), (x,), dy)
    assert torch.equal(got, want)


@pytest.mark.parametrize("which", range(1, 8))
def test_workspace_of_the_wanted_gradients(which, monkeypatch):
    """dg | du and parts of K are dx's and dw13's; dw2 alone takes nothing."""
    t, h, i = 40, 64, 48
    x, w13, w2, dy = D.ffn_inputs(t, h, i, 0, device="cpu")
    calls = []
    monkeypatch.setattr(L, "moe_ffn_backward", lambda *args: calls.append(args))
    monkeypatch.setattr(ffn, "current_raw_stream", lambda index: 0)
    dx, dw13, dw2 = (v if which >> k & 1 else None for k, v in enumerate((x, w13, w2)))
    ffn._backward(dy, x, w13, w2, None, None, dx, dw13, dw2, L.MOE_TYPE_BF16, 0)
    workspace, ws_bytes = calls[0][-3:-1]
    assert ws_bytes == (0 if which == 4 else L.moe_ffn_workspace_query(t, h, i)[1]) and bool(workspace) == bool(ws_bytes)


@pytest.mark.gpu
@pytest.mark.parametrize("t,h,i", [(3, 72, 40), (1000, 128, 2048)])
def test_dw2_alone_without_a_workspace(t, h, i):
    x, w13, w2, dy = D.ffn_inputs(t, h, i, 2)
    _, gu, hid = m.gated_ffn_forward(x, w13, w2)
    want, got = torch.empty_like(w2), torch.empty_like(w2)
    m.gated_ffn_backward(dy, x, w13, w2, gu, hid, dx=torch.empty_like(x), dw2=want)
    L.moe_ffn_backward(dy.data_ptr(), dy.stride(0), 0, 0, 0, 0, 0, hid.data_ptr(), t, h, i, 0, 0, 0, got.data_ptr(),
                       L.MOE_TYPE_BF16, 0, 0, 0, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(got, want)
    got.zero_()
    m.gated_ffn_backward(dy, x, w13, w2, None, hid, dw2=got)
    assert torch.equal(got, want)
