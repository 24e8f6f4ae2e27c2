"""Derivatives that the gated block cannot give are refused, not left out."""

import pytest
import torch
import torch.autograd.forward_ad as fwd

import mixture_experts_ffn_route_amd as m
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
