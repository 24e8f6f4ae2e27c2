"""Derivatives that the gated block cannot give are refused, not left out."""

import pytest
import torch
import torch.autograd.forward_ad as fwd

import mixture_experts_ffn_route_amd as m
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
