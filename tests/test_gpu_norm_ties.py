"""e4m3 codes of the norm whose quotients lie in the middle of two codes.

y / scale is 448 p / max p with p = (x + residual) weight: the row's factor
cancels.  Short mantissas put one quotient in some thousands exactly in the
middle of two codes, where RNE takes the even one; FP32 arithmetic whose steps
are all exact has to find it.  A quotient that is not in a middle may go wrong
only within its six roundings (sum and product of p and of max p, 7/8 p, the
quotient): 6 half steps of float32.
"""

import numpy as np
import pytest
import torch

from oracle import formats
from tests.test_gpu_norm import U, _inputs

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_ffn_route_amd import rms_norm_quant


def _f32(v):
    return v.astype(np.float32).astype(np.float64) == v


def _reference(x, r, w, T, H):
    """Quotients in float64 (exact in the middle of two codes), and whether
    every step of theirs is exact in float32."""
    s = x.double().cpu().numpy() + (0 if r is None else r.double().cpu().numpy())
    p = (s * w.double().cpu().numpy()).reshape(T, H // 128, 128)
    top = np.abs(p).max(axis=2, keepdims=True)
    short = _f32(s).reshape(p.shape) & _f32(p) & _f32(0.875 * p)
    at = np.abs(p).argmax(axis=2)[:, :, None]
    return p * 448.0 / top, short & np.take_along_axis(short, at, axis=2)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rtype,wtype", [(None, torch.bfloat16), (torch.bfloat16, torch.bfloat16),
                                         (torch.bfloat16, torch.float32), (None, torch.float32)])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -40, 2.0 ** 60])
def test_quotients_in_the_middle(rtype, wtype, scale, bf16):
    T, H = 512, 4096
    x, r, w = _inputs(T, H, rtype, wtype, 23)
    x = (scale * x.float()).bfloat16()
    r = None if r is None else (scale * r.float()).to(rtype)
    q, short = _reference(x, r, w, T, H)
    got = rms_norm_quant(x, w, r, eps=0.0, bf16=bf16).codes.cpu().numpy().view(np.uint8).reshape(q.shape)
    want = formats.e4m3_encode_rne_sat(q)
    lo, hi = formats.e4m3_encode_rne_sat(q * (1 - 6 * U)), formats.e4m3_encode_rne_sat(q * (1 + 6 * U))
    middle = (lo != hi) & short & (np.abs(q) < 448)
    if wtype == torch.bfloat16:
        assert middle.sum() > 100
    wrong = got != want
    assert not np.any(wrong & middle), f"{np.sum(wrong & middle)} of {middle.sum()} exact quotients"
    assert np.all(~wrong | (lo != hi)) and wrong.sum() <= 32


@pytest.mark.parametrize("wtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size,wsize", [(1e30, 1e10), (1e-30, 1e-12), (1e5, 1e33)])
def test_fp32_residual_beyond_the_range_of_its_products(size, wsize, wtype):
    """x + residual times the weight leaves float32's range, y does not: the
    codes from 2^-6 up are those of 64-bit arithmetic there too."""
    T, H = 128, 4096
    x, r, w = _inputs(T, H, torch.float32, wtype, 29, scale=size)
    w = (w.float() * wsize).to(wtype)
    q, _ = _reference(x, r, w, T, H)
    got = rms_norm_quant(x, w, r, eps=0.0).codes.cpu().numpy().view(np.uint8).reshape(q.shape)
    want = formats.e4m3_encode_rne_sat(q)
    seen = np.abs(q) >= 2.0 ** -6
    assert np.array_equal(got[seen], want[seen])
