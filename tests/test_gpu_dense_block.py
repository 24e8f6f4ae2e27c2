"""The dense products where a decoder layer uses them: behind the norm, and as
the shared expert of a MoE block."""

import pytest
import torch

from tests import dense_util as D
from tests.test_gpu_block import _make

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_ffn_route_amd import MoEBlock, MoESharedExpert, fp8_matmul, gated_ffn, rms_norm_quant


def _shared(H, I, seed):
    _, _, w13, s13 = D.fp8_inputs(1, 2 * I, H, seed)
    _, _, w2, s2 = D.fp8_inputs(1, H, I, seed + 1)
    return MoESharedExpert(w13, s13, w2, s2)


@pytest.mark.parametrize("mx", [False, "e4m3"])
@pytest.mark.parametrize("T", [1, 9, 17, 70, 300])
def test_block_with_a_shared_expert(T, mx):
    _, _, _, weight, block, x, r = _make(T, mx, seed=T)
    shared = _shared(1024, 512, T)
    both = MoEBlock(weight, block.router, block.layer, shared=shared)
    routed, res = block.forward(x, r)
    out, res2 = both.forward(x, r)
    n = rms_norm_quant(x, weight, r, bf16=True)
    want, bound = D.shared64(n.codes, n.scale, shared.w13, shared.w13_scale, shared.w2, shared.w2_scale, routed)
    D.assert_within(out, want, bound, f"T={T}")
    assert torch.equal(res, res2)
    given = torch.empty_like(out)
    got, _ = both.forward(x, r, out=given)
    assert got is given and torch.equal(given, out)


def test_block_with_a_shared_expert_captured_and_replayed():
    for T in (5, 90):
        _, _, _, weight, block, x, r = _make(T, False, seed=T)
        both = MoEBlock(weight, block.router, block.layer, shared=_shared(1024, 512, 3))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            both.forward(x, r)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out, _ = both.forward(x, r)
        torch.cuda.synchronize()
        for seed in (1, 2, 3):
            g = torch.Generator(device="cuda").manual_seed(seed)
            x.copy_(torch.randn(T, 1024, generator=g, device="cuda").bfloat16())
            want, _ = both.forward(x, r)
            out.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_block_refuses_a_shared_expert_of_another_width():
    _, _, _, weight, block, _, _ = _make(2, False)
    with pytest.raises(ValueError, match="shared"):
        MoEBlock(weight, block.router, block.layer, shared=_shared(512, 256, 0))


@pytest.mark.parametrize("T", [1, 30, 200])
def test_norm_then_product(T):
    """A projection of the norm's rows, its result onto the residual."""
    H, N = 1024, 1024
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    r = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    weight = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16()
    _, _, w, ws = D.fp8_inputs(1, N, H, 4)
    n = rms_norm_quant(x, weight, r)
    residual = n.residual.clone()
    out = fp8_matmul(n.codes, n.scale, w, ws, add=n.residual, out=n.residual)
    want, bound = D.rounded(*D.product64(n.codes, n.scale, w, ws), residual)
    D.assert_within(out, want, bound, f"T={T}")


def test_shared_expert_of_a_trained_block():
    """The BF16 block's weights, quantised, as a shared expert: its output is
    that of the quantised weights and rows, and near the BF16 block's."""
    T, H, I = 200, 512, 256
    x, w13, w2, _ = D.ffn_inputs(T, H, I, 5)
    y = gated_ffn(x, w13, w2)
    (q13, s13), (q2, s2), (qx, sx) = D.quantise(w13, 128), D.quantise(w2, 128), D.quantise(x, 1)
    out = MoESharedExpert(q13, s13, q2, s2).forward(qx, sx)
    want, bound = D.shared64(qx, sx, q13, s13, q2, s2)
    D.assert_within(out, want, bound, "quantised")
    # e4m3 keeps 4 bits: half a step is 2^-4 of a value at most, 2^-4 / sqrt(3) in
    # the mean; it meets x, w13 (with g and u both), h and w2: 6 times, slopes to 1.1
    assert D.rel_rms(out, y.double()) < 6 ** 0.5 * 1.1 * 2.0 ** -4 / 3 ** 0.5
