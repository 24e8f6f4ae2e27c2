"""The layer for a few tokens (moe_layer_decode) against the float64 oracle and
against stage + forward.

The outputs are held to the layer's own parity rule (parity_util: relative
Frobenius error 1e-2, 99.9% of the elements within 5e-2 of their row's RMS),
which covers e4m3 codes of h that fall on the other side of a tie; what does
not depend on rounding (masked rows, status bits, repeated calls, rows that
must not change) is compared for equality.
"""

import numpy as np
import pytest
import torch

from oracle import moe_ref
from synthetic import MoEShape, make_layer_inputs
from tests.parity_util import assert_output_close

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_ffn_route_amd import MoEError, _lib as L
    from mixture_experts_ffn_route_amd.harness import make_layer, run_forward, to_device


def _bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def _oracle(inp, idx=None, w=None, **kw):
    return moe_ref.forward_fp8(inp.x_bf16, inp.topk_idx if idx is None else idx, inp.topk_w if w is None else w,
                               inp.w13, inp.w13_scale, inp.w2, inp.w2_scale, **kw)


def _setup(T, H, I, E, K, seed=0, masked=0.0, max_rows=None, **kw):
    shape = MoEShape(T, H, I, E, K, "topk")
    inp = make_layer_inputs(shape, seed=seed, masked_fraction=masked)
    dev = to_device(inp)
    return inp, dev, make_layer(shape, dev, max_rows=max_rows, **kw)


@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 15, 16])
@pytest.mark.parametrize("H,I,E,K", [(256, 128, 8, 2), (2048, 768, 32, 6), (1152, 384, 16, 8)])
def test_matches_oracle_and_forward(T, H, I, E, K):
    inp, dev, layer = _setup(T, H, I, E, K, seed=T)
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    got = layer.decode(dev.x, dev.topk_idx, dev.topk_w, status=status)
    res = _oracle(inp)
    assert_output_close(_bits(got), res.out_bits, f"decode T={T}")
    assert int(status) == res.status == 0
    assert_output_close(_bits(got), _bits(run_forward(layer, dev)), "forward")


@pytest.mark.parametrize("T,H,I,E,K", [
    (1, 128, 128, 1, 1),          # one K-block: seven of the eight waves have none
    (16, 128, 128, 1, 1),         # every token at one expert
    (4, 384, 128, 3, 2),          # output rows that end inside a 256-row weight tile
    (7, 896, 256, 5, 4),          # K-blocks that do not divide by the waves
    (16, 256, 256, 200, 8),       # 128 routes over many experts
    (2, 16384, 128, 4, 2), (2, 128, 16384, 4, 2),  # the longest rows
])
def test_odd_shapes(T, H, I, E, K):
    inp, dev, layer = _setup(T, H, I, E, K, seed=3)
    got = layer.decode(dev.x, dev.topk_idx, dev.topk_w)
    assert_output_close(_bits(got), _oracle(inp).out_bits, "decode")


@pytest.mark.parametrize("T,masked", [(1, 1.0), (5, 0.3), (16, 0.8), (16, 1.0)])
def test_masked_routes(T, masked):
    """The generator masks routes with NaN and infinite weights and leaves the
    last token none: its row is +0."""
    inp, dev, layer = _setup(T, 512, 256, 16, 4, seed=1, masked=masked)
    out = torch.full((T + 2, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    layer.decode(dev.x, dev.topk_idx, dev.topk_w, out=out[:T], status=status)
    res = _oracle(inp)
    assert_output_close(_bits(out[:T]), res.out_bits, "masked")
    assert np.all(_bits(out[T - 1]) == 0) and int(status) == res.status
    assert torch.all(out[T:] == 3.0)


def test_route_checks():
    """Ids out of range, repeated ids and weights that are no numbers are
    masked and reported, as in stage + forward."""
    inp, dev, layer = _setup(6, 512, 256, 16, 4, seed=2)
    idx, w = inp.topk_idx.copy(), inp.topk_w.copy()
    idx[0] = [3, 3, 5, 3]
    idx[1, 2] = 16
    idx[2, 0] = -7
    idx[3] = [9, 9, 9, 9]
    w[3, 0] = np.nan          # the first of the four stays in its place, and is then masked
    w[4, 1] = np.inf
    dev.topk_idx, dev.topk_w = torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = layer.decode(dev.x, dev.topk_idx, dev.topk_w, status=status)
    res = _oracle(inp, idx, w)
    assert int(status) == res.status == (L.MOE_DEV_BAD_EXPERT | L.MOE_DEV_DUPLICATE | L.MOE_DEV_NONFINITE)
    assert_output_close(_bits(got), res.out_bits, "checks")
    assert np.all(_bits(got[3]) == 0)
    layer.decode(dev.x[4:5], dev.topk_idx[5:6], dev.topk_w[5:6], status=status)
    assert int(status) == 0   # the next call's own bits


def test_repeated_ids_without_checks():
    """Without route checks a repeated id counts as often as it is given."""
    inp, dev, layer = _setup(3, 512, 256, 16, 4, seed=4, flags=0)
    idx = inp.topk_idx.copy()
    idx[1] = [2, 7, 2, 2]
    dev.topk_idx = torch.from_numpy(idx).cuda()
    got = layer.decode(dev.x, dev.topk_idx, dev.topk_w)
    assert_output_close(_bits(got), _bits(run_forward(layer, dev)), "repeated")


def test_prequantised_rows_give_the_same_bits():
    inp, dev, layer = _setup(9, 1024, 384, 16, 4, seed=5)
    want = layer.decode(dev.x, dev.topk_idx, dev.topk_w)
    layer.stage(dev.x, dev.topk_idx, dev.topk_w)
    codes = layer.region("xq", torch.uint8, (9, 1024)).clone()
    scales = layer.region("xs", torch.float32, (9, 8)).clone()
    got = layer.decode(codes, dev.topk_idx, dev.topk_w, x_scale=scales)
    assert torch.equal(got, want)


def test_scales_beyond_float32_products():
    """Activation scales from 2^-100 to 2^60 against weight scales of the
    opposite size: only the product of the two is ordinary."""
    inp, dev, layer0 = _setup(5, 512, 256, 8, 2, seed=6)
    for p in (-100, 60):
        d = to_device(inp)
        x = torch.ldexp(dev.x.float(), torch.tensor(float(p), device="cuda")).bfloat16()
        d.w13_scale = torch.ldexp(dev.w13_scale, torch.tensor(float(-p), device="cuda"))
        layer = make_layer(inp.shape, d)
        assert torch.equal(layer.decode(x, dev.topk_idx, dev.topk_w), layer0.decode(dev.x, dev.topk_idx, dev.topk_w))


def test_bad_rows_touch_no_other():
    inp, dev, layer = _setup(6, 512, 256, 4, 2, seed=7)
    want = layer.decode(dev.x, dev.topk_idx, dev.topk_w)
    for bad in (float("nan"), float("inf")):
        x = dev.x.clone()
        x[2, 300] = bad
        got = layer.decode(x, dev.topk_idx, dev.topk_w)
        keep = [0, 1, 3, 4, 5]
        assert torch.equal(got[keep], want[keep]) and torch.isnan(got[2]).all()
    assert torch.equal(layer.decode(dev.x, dev.topk_idx, dev.topk_w), want)  # nothing is left behind


def test_repeated_calls_and_the_staged_batch():
    inp, dev, layer = _setup(12, 1024, 384, 32, 8, seed=8, max_rows=64)
    staged = layer.stage(dev.x, dev.topk_idx, dev.topk_w)
    want = layer.decode(dev.x, dev.topk_idx, dev.topk_w)
    for T in (12, 1, 7, 12):
        part = layer.decode(dev.x[:T], dev.topk_idx[:T], dev.topk_w[:T])
        assert_output_close(_bits(part), _bits(want[:T]), f"first {T}")
    layer.forward()  # the batch staged before the calls
    first = staged.clone()
    layer.stage(dev.x, dev.topk_idx, dev.topk_w, out=staged)
    layer.forward()
    assert torch.equal(staged, first)
    for _ in range(5):
        assert torch.equal(layer.decode(dev.x, dev.topk_idx, dev.topk_w), want)


def test_capacity_does_not_drop_routes():
    inp, dev, layer = _setup(8, 512, 256, 16, 4, seed=9, capacity_factor=0.25)
    assert_output_close(_bits(layer.decode(dev.x, dev.topk_idx, dev.topk_w)), _oracle(inp).out_bits, "capacity")


def test_stream_and_graph_replays():
    inp, dev, layer = _setup(4, 1024, 384, 16, 4, seed=10)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x, idx, w = dev.x.clone(), dev.topk_idx.clone(), dev.topk_w.clone()
    out = torch.empty_like(x)
    with torch.cuda.stream(side):
        layer.decode(x, idx, w, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            layer.decode(x, idx, w, out=out)
    torch.cuda.synchronize()
    for seed in (1, 2, 3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(4, 1024, generator=g, device="cuda").bfloat16())
        idx.copy_(torch.rand(4, 16, generator=g, device="cuda").topk(4, dim=1).indices.int())
        want = layer.decode(x, idx, w)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def _setup_mx(T, H, I, E, K, elem, seed=0, masked=0.0):
    shape = MoEShape(T, H, I, E, K, "topk")
    inp = make_layer_inputs(shape, seed=seed, masked_fraction=masked,
                            weight_format="mxfp8" if elem == "e4m3" else "mxfp8_e5m2")
    dev = to_device(inp)
    return inp, dev, make_layer(shape, dev, mx=elem)


def _oracle_mx(inp, elem):
    return moe_ref.forward_mx(inp.x_bf16, inp.topk_idx, inp.topk_w, inp.w13, inp.w13_scale, inp.w2, inp.w2_scale,
                              elem=elem)


@pytest.mark.parametrize("elem", ["e4m3", "e5m2"])
@pytest.mark.parametrize("T,H,I,E,K,masked", [
    (1, 2048, 768, 32, 6, 0.0), (5, 2048, 768, 32, 6, 0.3), (16, 1152, 384, 16, 8, 0.0), (3, 128, 128, 1, 1, 0.0),
    (4, 384, 128, 3, 2, 0.0), (9, 896, 256, 5, 4, 0.5), (2, 16384, 128, 4, 2, 0.0), (2, 128, 16384, 4, 2, 0.0),
    (16, 256, 256, 16, 4, 1.0)])
def test_mxfp8_weights(T, H, I, E, K, masked, elem):
    inp, dev, layer = _setup_mx(T, H, I, E, K, elem, seed=T, masked=masked)
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    got = layer.decode(dev.x, dev.topk_idx, dev.topk_w, status=status)
    res = _oracle_mx(inp, elem)
    assert_output_close(_bits(got), res.out_bits, f"mx {elem}")
    assert int(status) == res.status
    assert_output_close(_bits(got), _bits(run_forward(layer, dev)), "forward")


def test_mxfp8_exponents_of_any_size():
    """Weight exponents 60 and -70 away from the usual against activations of
    the opposite size: widening is exact, so nothing changes."""
    inp, dev, layer0 = _setup_mx(5, 512, 256, 8, 2, "e4m3", seed=6)
    want = layer0.decode(dev.x, dev.topk_idx, dev.topk_w)
    for p in (-60, 70):
        d = to_device(inp)
        x = torch.ldexp(dev.x.float(), torch.tensor(float(p), device="cuda")).bfloat16()
        d.w13_scale = (dev.w13_scale.int() - p).to(torch.uint8)
        layer = make_layer(inp.shape, d, mx=True)
        assert torch.equal(layer.decode(x, dev.topk_idx, dev.topk_w), want)


def test_mxfp8_bad_rows_touch_no_other():
    inp, dev, layer = _setup_mx(6, 512, 256, 4, 2, "e4m3", seed=7)
    want = layer.decode(dev.x, dev.topk_idx, dev.topk_w)
    x = dev.x.clone()
    x[2, 300] = float("nan")
    got = layer.decode(x, dev.topk_idx, dev.topk_w)
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(got[keep], want[keep]) and torch.isnan(got[2]).all()
    with pytest.raises(MoEError):   # codes are for the FP8 path
        layer.decode(torch.zeros(6, 512, dtype=torch.uint8, device="cuda"), dev.topk_idx, dev.topk_w,
                     x_scale=torch.ones(6, 4, device="cuda"))


def test_no_tokens_and_refusals():
    inp, dev, layer = _setup(16, 256, 128, 8, 2, seed=11, max_rows=32)
    status = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    out = layer.decode(dev.x[:0], dev.topk_idx[:0], dev.topk_w[:0], status=status)
    assert out.shape == (0, 256) and int(status) == 0
    x17 = torch.zeros(17, 256, dtype=torch.bfloat16, device="cuda")
    i17, w17 = torch.zeros(17, 2, dtype=torch.int32, device="cuda"), torch.zeros(17, 2, device="cuda")
    with pytest.raises(MoEError) as ei:
        layer.decode(x17, i17, w17)
    assert ei.value.status == L.MOE_ERR_CAPACITY
    for args in ((dev.x.float(), dev.topk_idx, dev.topk_w), (dev.x[:, :128], dev.topk_idx, dev.topk_w),
                 (dev.x, dev.topk_idx.long(), dev.topk_w), (dev.x, dev.topk_idx, dev.topk_w.double()),
                 (dev.x, dev.topk_idx[:3], dev.topk_w), (dev.x.cpu(), dev.topk_idx, dev.topk_w)):
        with pytest.raises(ValueError):
            layer.decode(*args)
    with pytest.raises(ValueError):
        layer.decode(dev.x.view(torch.uint8)[:, :256].contiguous(), dev.topk_idx, dev.topk_w)  # codes without scales
    small = make_layer(MoEShape(4, 256, 128, 8, 2, "topk"), dev, max_rows=4)
    with pytest.raises(MoEError):
        small.decode(dev.x[:5], dev.topk_idx[:5], dev.topk_w[:5])


def test_full_size():
    """A DeepSeek-V3-like share, every expert reached."""
    inp, dev, layer = _setup(16, 7168, 2048, 32, 8, seed=12)
    got = layer.decode(dev.x, dev.topk_idx, dev.topk_w)
    assert_output_close(_bits(got), _oracle(inp).out_bits, "full size")
    one = layer.decode(dev.x[:1], dev.topk_idx[:1], dev.topk_w[:1])
    # sums are split over waves by the batch's experts: the same row to a rounding of float32
    assert_output_close(_bits(one), _bits(got[:1]), "one token of the batch")
