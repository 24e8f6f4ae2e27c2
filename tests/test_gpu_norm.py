"""Residual RMS norm with e4m3 rows (moe_rms_norm_quant) against its formula
in float64.

Bounds, u = 2^-24 the half step of float32: s = x + r is one rounding (u);
the factor 1/sqrt(mean + eps) comes from float64 (u); y = s * f * w adds two
roundings, so y is within 4u (taken as 5u for the second-order terms).  A
scale is one more (max|y| / 448): 6u.  A quotient y / scale adds its own
rounding: within 12u.  The outputs then add half a step of their own type:
2^-8 for bfloat16, and for a code the nearest e4m3 value of a quotient within
12u of the formula's.
"""

import numpy as np
import pytest
import torch

from oracle import formats

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_ffn_route_amd import MoEError, NormOutput, rms_norm_quant

U = 2.0 ** -24
BF16 = 2.0 ** -8


def _formula(x, r, w, eps):
    s = x.double().cpu().numpy()
    if r is not None:
        s = s + r.double().cpu().numpy()
    with np.errstate(all="ignore"):
        y = s / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps) * w.double().cpu().numpy()
    return s, y


def _check(got, x, r, w, eps, bf16):
    s, y = _formula(x, r, w, eps)
    T, H = s.shape
    if r is not None:
        half = BF16 if r.dtype == torch.bfloat16 else 0.0
        assert got.residual.dtype == r.dtype
        assert np.all(np.abs(got.residual.double().cpu().numpy() - s) <= (half + 2 * U) * np.abs(s))
    if bf16:
        err = np.abs(got.y.double().cpu().numpy() - y)
        # half a step of a bfloat16 below 2^-126 is 2^-134
        assert np.all(err <= (BF16 + 5 * U) * np.abs(y) + 2.0 ** -134)
    if got.codes is None:
        return
    b = y.reshape(T, H // 128, 128)
    scale = np.abs(b).max(axis=2) / 448.0
    gs = got.scale.double().cpu().numpy()
    assert np.all(np.abs(gs - scale) <= 6 * U * scale + 2.0 ** -149)
    codes = got.codes.cpu().numpy().view(np.uint8).reshape(T, H // 128, 128)
    big = scale >= 2.0 ** -120  # smaller scales are subnormal: their own step is what counts
    q = b / np.where(scale > 0, scale, 1.0)[:, :, None]
    lo = formats.e4m3_encode_rne_sat(q * (1 - 12 * U))
    hi = formats.e4m3_encode_rne_sat(q * (1 + 12 * U))
    ok = (codes == lo) | (codes == hi) | ((q == 0) & ((codes & 0x7f) == 0))
    assert np.all(ok | ~big[:, :, None])
    assert np.all(codes[scale == 0] & 0x7f == 0)


def _inputs(T, H, rtype, wtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (scale * torch.randn(T, H, generator=g, device="cuda")).bfloat16()
    r = None if rtype is None else (2 * scale * torch.randn(T, H, generator=g, device="cuda")).to(rtype)
    w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(wtype)
    return x, r, w


@pytest.mark.parametrize("wtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [2048, 7168])
@pytest.mark.parametrize("in_place", [False, True])
def test_codes_are_those_of_64_bits(H, wtype, in_place):
    """FP32 residual: a few of a million quotients lie closer to the middle of
    two codes than FP32 can tell.  The factor 1/sqrt(mean + eps) cancels in
    y / scale, so the formula's own rounding is a few 2^-53.  Codes below
    2^-6 may go by FP32's quotient."""
    T = 2 ** 21 // H
    x, r, w = _inputs(T, H, torch.float32, wtype, 17)
    b = _formula(x, r, w, 1e-6)[0] * w.double().cpu().numpy()
    q = b.reshape(T, H // 128, 128) * 448.0
    q = q / (np.abs(q).max(axis=2, keepdims=True) / 448.0)
    want = formats.e4m3_encode_rne_sat(q)
    out = None
    if in_place:  # the new residual over the old one, the BF16 rows over x
        out = NormOutput(torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, H // 128, device="cuda"),
                         x, r)
    got = rms_norm_quant(x, w, r, out=out)
    codes = got.codes.cpu().numpy().view(np.uint8).reshape(want.shape)
    assert np.array_equal(codes[np.abs(q) >= 2.0 ** -6], want[np.abs(q) >= 2.0 ** -6])


@pytest.mark.parametrize("rtype", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("wtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 128), (3, 256), (1, 7168), (37, 7168), (5, 8192), (4, 8320), (2, 16384),
                                 (301, 2048), (1100, 640)])
def test_norm_matches_formula(T, H, rtype, wtype):
    x, r, w = _inputs(T, H, rtype, wtype, T * 7 + H)
    got = rms_norm_quant(x, w, r, bf16=True)
    _check(got, x, r, w, 1e-6, True)
    # the codes alone, and the BF16 rows alone, are the same
    only = rms_norm_quant(x, w, r)
    assert only.y is None and torch.equal(only.codes, got.codes) and torch.equal(only.scale, got.scale)
    rows = rms_norm_quant(x, w, r, codes=False, bf16=True)
    assert rows.codes is None and rows.scale is None and torch.equal(rows.y, got.y)


def test_more_rows_than_workgroups():
    """A launch has at most 65536 workgroups; later rows are their second turn."""
    T = 65536 + 129
    x, r, w = _inputs(T, 128, torch.bfloat16, torch.bfloat16, 5)
    _check(rms_norm_quant(x, w, r, bf16=True), x, r, w, 1e-6, True)


def test_no_tokens():
    x, r, w = _inputs(0, 256, torch.bfloat16, torch.bfloat16, 1)
    got = rms_norm_quant(x, w, r)
    assert got.codes.shape == (0, 256) and got.scale.shape == (0, 2) and got.residual.shape == (0, 256)


@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e18, 1e30])
def test_row_sizes_beyond_float32_squares(scale):
    """Squares of such rows leave float32's range; the sum is kept in float64."""
    x, r, w = _inputs(6, 512, torch.float32, torch.float32, 3, scale=scale)
    _check(rms_norm_quant(x, w, r, eps=0.0, bf16=True), x, r, w, 0.0, True)


def test_zero_rows_blocks_and_eps():
    x, _, w = _inputs(4, 512, None, torch.float32, 9)
    x[1] = 0
    x[2, 128:256] = 0
    got = rms_norm_quant(x, w, bf16=True, eps=1e-5)
    _check(got, x, None, w, 1e-5, True)
    assert not got.scale[1].any() and not got.codes[1].any() and got.scale[2, 1] == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_rows_stay_visible(bad):
    """A NaN or an infinity makes every value that depends on it NaN after
    dequantisation, and no other row."""
    x, r, w = _inputs(3, 384, torch.bfloat16, torch.bfloat16, 2)
    clean = rms_norm_quant(x, w, r, bf16=True)
    x[1, 5] = bad
    got = rms_norm_quant(x, w, r, bf16=True)
    deq = got.codes.view(torch.float8_e4m3fn).float().view(3, 3, 128) * got.scale[..., None]
    assert torch.isnan(got.y[1, 5]) and torch.isnan(deq[1, 0, 5])
    for t in (0, 2):
        assert torch.equal(got.codes[t], clean.codes[t]) and torch.equal(got.y[t], clean.y[t])


def test_strides_and_in_place():
    T, H = 19, 1024
    x0, r0, w = _inputs(T, H, torch.bfloat16, torch.bfloat16, 4)
    want = rms_norm_quant(x0, w, r0, bf16=True)
    wide = torch.full((T, 2 * H + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    x, r = wide[:, :H], wide[:, H + 8:]
    x.copy_(x0)
    r.copy_(r0)
    out = NormOutput(torch.empty(T, H, dtype=torch.uint8, device="cuda"),
                     torch.empty(T, H // 128, device="cuda"), None, r)
    got = rms_norm_quant(x, w, r, out=out)  # the residual is updated where it stands
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scale, want.scale)
    assert torch.equal(r, want.residual) and torch.equal(x, x0)
    assert torch.all(wide[:, H:H + 8] == 7.0)
    # y over x itself
    xc, rc = x0.clone(), r0.clone()
    got = rms_norm_quant(xc, w, rc, out=NormOutput(None, None, xc, rc))
    assert torch.equal(xc, want.y) and torch.equal(rc, want.residual)


def test_stream_and_graph_replays():
    T, H = 33, 2048
    x, r, w = _inputs(T, H, torch.bfloat16, torch.float32, 6)
    want = rms_norm_quant(x, w, r, bf16=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = NormOutput(*(torch.zeros_like(t) for t in want))
    with torch.cuda.stream(side):
        rms_norm_quant(x, w, r, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            rms_norm_quant(x, w, r, out=out)
    torch.cuda.synchronize()
    for seed in (7, 8, 9):
        x2, r2, _ = _inputs(T, H, torch.bfloat16, torch.float32, seed)
        x.copy_(x2)
        r.copy_(r2)
        eager = rms_norm_quant(x2, w, r2, bf16=True)
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)


def test_rows_feed_the_layer():
    """The rows and scales are what the layer's staging takes as prequantised."""
    from mixture_experts_ffn_route_amd.harness import make_layer, to_device
    from synthetic import CONFIGS, make_layer_inputs
    shape = CONFIGS["tiny"]
    inp = make_layer_inputs(shape, seed=3)
    dev = to_device(inp)
    layer = make_layer(shape, dev)
    _, r, w = _inputs(shape.tokens, shape.hidden, torch.bfloat16, torch.bfloat16, 12)
    n = rms_norm_quant(dev.x, w, r)
    out = layer.stage(n.codes, dev.topk_idx, dev.topk_w, x_scale=n.scale)
    layer.forward()
    assert torch.equal(layer.region("xq", torch.uint8, (shape.tokens, shape.hidden)), n.codes)
    assert torch.equal(layer.region("xs", torch.float32, (shape.tokens, shape.hidden // 128)), n.scale)
    assert torch.isfinite(out.float()).all() and layer.status() == 0


def test_refusals():
    x, r, w = _inputs(4, 256, torch.bfloat16, torch.bfloat16, 1)
    for args in ((x.float(), w, r), (x, w.half(), r), (x, w[:128], r), (x, w, r[:3]), (x, w, r.half()),
                 (x.t().contiguous().t(), w, r), (x.cpu(), w, r), (x, w.cpu(), r), (x[0], w, None)):
        with pytest.raises(ValueError):
            rms_norm_quant(*args)
    with pytest.raises(ValueError):
        rms_norm_quant(x, w, out=NormOutput(None, None, torch.empty_like(x), torch.empty_like(x)))
    with pytest.raises(MoEError):
        rms_norm_quant(x, w, codes=False)                       # nothing wanted
    with pytest.raises(MoEError):
        rms_norm_quant(x, w, eps=-1.0)
    with pytest.raises(MoEError):
        rms_norm_quant(x[:, :200].contiguous(), w[:200].contiguous())  # not whole blocks
    with pytest.raises(MoEError):
        rms_norm_quant(x[:1].expand(4, 256), w)                 # rows on top of each other
    with pytest.raises(MoEError):
        rms_norm_quant(torch.zeros(4, 260, dtype=torch.bfloat16, device="cuda")[:, 4:260], w)  # 8-byte rows
