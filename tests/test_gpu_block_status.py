"""MoEBlock means the same on both sides of its few-token limit: what it
reports, and which routes it drops."""

import pytest
import torch

from tests.test_gpu_block import _make

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_ffn_route_amd import MoEBlock, _lib as L
    from mixture_experts_ffn_route_amd.harness import make_layer, to_device


@pytest.mark.parametrize("mx", [False, "e4m3"])
@pytest.mark.parametrize("T", [1, 5, 9, 20])
def test_status_word(T, mx):
    """A NaN in a token: its routing weights are masked and reported."""
    _, _, _, _, block, x, r = _make(T, mx, base=0, seed=T)
    # the router's lowest experts, which a row of NaN takes, are this GPU's
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    bad = x.clone()
    bad[T - 1, 7] = float("nan")
    out, _ = block.forward(bad, r, status=status)
    assert int(status) == L.MOE_DEV_NONFINITE
    clean, _ = block.forward(x, r, status=status)
    assert int(status) == 0
    assert torch.equal(out[:T - 1], clean[:T - 1])
    block.forward(bad, r)   # no word given
    assert int(status) == 0


@pytest.mark.parametrize("T", [2, 8])
def test_a_layer_that_may_drop_routes(T):
    """The same routes are dropped and reported as in stage + forward."""
    from synthetic import MoEShape, make_layer_inputs
    _, _, _, weight, full, x, r = _make(T, False, base=0, seed=T)
    inp = make_layer_inputs(MoEShape(T, 1024, 384, 16, 4, "topk"), seed=T)
    small = make_layer(inp.shape, to_device(inp), capacity_factor=0.125)
    block = MoEBlock(weight, full.router, small)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, _ = block.forward(x, r, status=status)
    from mixture_experts_ffn_route_amd import rms_norm_quant
    n = rms_norm_quant(x, weight, r, bf16=True)
    idx, w = full.router.route(n.y)
    want = small.stage(n.codes, idx, w, x_scale=n.scale)
    small.forward()
    assert torch.equal(out, want) and int(status) == small.status() == L.MOE_DEV_CAPACITY


@pytest.mark.parametrize("T", [4, 30])
def test_status_word_of_a_captured_call(T):
    _, _, _, _, block, x, r = _make(T, False, base=0, seed=T)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    good, bad = x.clone(), x.clone()
    bad[0, 3] = float("inf")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.forward(x, r, status=status)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out, _ = block.forward(x, r, status=status)
    torch.cuda.synchronize()
    for rows, bits in ((good, 0), (bad, L.MOE_DEV_NONFINITE), (good, 0), (bad, L.MOE_DEV_NONFINITE)):
        x.copy_(rows)
        eager = torch.full_like(status, -1)
        want, _ = block.forward(x, r, status=eager)
        out.zero_()
        status.fill_(-1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[1:], want[1:]) and int(status) == int(eager) == bits


def test_status_word_is_checked():
    _, _, _, _, block, x, r = _make(20, False)
    for bad in (torch.zeros(1, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"),
                torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(ValueError):
            block.forward(x, r, status=bad)
