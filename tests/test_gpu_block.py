"""Norm, router and layer run together (MoEBlock), as a decoder layer uses
them, against the same steps in float64.

The norm's rows are checked by themselves (test_gpu_norm) and taken as the
block makes them, since the experts they choose have to be equal; routing and
the experts' part follow from them.  The output is held to the layer's parity
rule.
"""

import numpy as np
import pytest
import torch

from oracle import formats, moe_ref
from synthetic import MoEShape, make_layer_inputs
from tests.parity_util import assert_output_close
from tests.test_gpu_router import reference

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_ffn_route_amd import MoEBlock, MoERouter, rms_norm_quant
    from mixture_experts_ffn_route_amd.harness import make_layer, to_device


def _bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def _make(T, mx, base=8, seed=0):
    """32 experts in 4 groups, 16 of them (from `base` on) on this GPU."""
    H, I, local, K = 1024, 384, 16, 4
    shape = MoEShape(T, H, I, local, K, "topk")
    inp = make_layer_inputs(shape, seed=seed, weight_format="mxfp8" if mx else "fp8_block")
    dev = to_device(inp)
    g = torch.Generator(device="cuda").manual_seed(seed)
    gate = (torch.randn(32, H, generator=g, device="cuda") * H ** -0.5).bfloat16()
    bias = 0.05 * torch.randn(32, generator=g, device="cuda")
    router = MoERouter(gate, K, max_rows=T, score="sigmoid", bias=bias, num_groups=4, top_groups=2, scale=1.5,
                       expert_base=base, local_experts=local)
    weight = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16()
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    r = torch.randn(T, H, generator=g, device="cuda")
    return inp, gate, bias, weight, MoEBlock(weight, router, make_layer(shape, dev, mx=mx)), x, r


def _experts(inp, mx, n, ids, w, base):
    """The experts' part in float64 from the norm's output ``n``."""
    E, H = inp.w13.shape[0], inp.w13.shape[2]
    if mx:
        x = n.y.double().cpu().numpy()
    else:
        x = moe_ref.dequant_rows_1x128(n.codes.cpu().numpy().view(np.uint8), n.scale.cpu().numpy())
    out = np.zeros((x.shape[0], H))
    for e in range(E):
        t, k = np.nonzero(ids - base == e)
        if t.size == 0:
            continue
        if mx:
            gu = x[t] @ moe_ref.dequant_mx(inp.w13[e], inp.w13_scale[e]).T
            h = moe_ref.silu(gu[:, :gu.shape[1] // 2]) * gu[:, gu.shape[1] // 2:]
            h = formats.bf16_bits_to_f64(formats.bf16_rne_bits(h))
            y = h @ moe_ref.dequant_mx(inp.w2[e], inp.w2_scale[e]).T
        else:
            _, codes, scales = moe_ref.fc1_swiglu_requant(x[t], inp.w13[e], inp.w13_scale[e])
            y = moe_ref.fc2(moe_ref.dequant_rows_1x128(codes, scales), inp.w2[e], inp.w2_scale[e])
        out[t] += w[t, k][:, None] * y
    return formats.bf16_rne_bits(out)


@pytest.mark.parametrize("mx", [False, "e4m3"])
@pytest.mark.parametrize("T", [1, 5, 6, 8, 9, 40])  # the few-token layer, and stage + forward
def test_block_matches_its_steps(T, mx):
    inp, gate, bias, weight, block, x, r = _make(T, mx, seed=T)
    out, res = block.forward(x, r)
    n = rms_norm_quant(x, weight, r, bf16=True)
    ids, w, _ = reference(n.y, gate, 4, "sigmoid", bias, 4, 2, scale=1.5)
    assert torch.equal(res, n.residual)
    assert_output_close(_bits(out), _experts(inp, mx, n, ids, w, 8), f"T={T}")


def test_block_without_local_experts():
    """No route of the batch is here: the block adds nothing."""
    inp, gate, bias, weight, block, x, r = _make(3, False, seed=1)
    ids = torch.empty(3, 4, dtype=torch.int32, device="cuda")
    n = rms_norm_quant(x, weight, r, bf16=True)
    block.router.route(n.y, ids=ids)
    away = [e for e in range(32) if e not in set(ids.flatten().tolist())]
    run = next((b for b in away if b + 1 in away), None)
    assert run is not None   # 12 routes leave 20 of 32 experts
    two = make_layer_inputs(MoEShape(3, 1024, 384, 4, 4, "topk"), seed=2)
    dev = to_device(two)
    router = MoERouter(gate, 4, max_rows=3, score="sigmoid", bias=bias, num_groups=4, top_groups=2,
                       expert_base=run, local_experts=2)
    idx, _ = router.route(n.y)
    assert (idx == -1).all()
    layer = make_layer(MoEShape(3, 1024, 384, 4, 4, "topk"), dev)
    w = torch.ones(3, 4, device="cuda")
    assert not layer.decode(n.codes, idx, w, x_scale=n.scale).any()


def test_block_captured_and_replayed():
    for T in (5, 24):
        _, _, _, _, block, x, r = _make(T, False, seed=T)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            block.forward(x, r)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out, res = block.forward(x, r)
        torch.cuda.synchronize()
        for seed in (1, 2, 3):
            g = torch.Generator(device="cuda").manual_seed(seed)
            x.copy_(torch.randn(T, 1024, generator=g, device="cuda").bfloat16())
            want, wres = block.forward(x, r)
            out.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(res, wres)


def test_block_refuses_parts_that_do_not_fit():
    _, gate, bias, weight, block, _, _ = _make(2, False)
    other = MoERouter(gate, 2, max_rows=2, local_experts=16)
    with pytest.raises(ValueError):
        MoEBlock(weight, other, block.layer)       # another top_k
    with pytest.raises(ValueError):
        MoEBlock(weight, MoERouter(gate, 4, max_rows=2), block.layer)   # 32 local experts for 16
