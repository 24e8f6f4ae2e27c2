"""Host-side refusals of moe_rms_norm_quant (no GPU: every bad call returns
before a launch)."""

import pytest

from mixture_experts_ffn_route_amd import _lib as L

GOOD = dict(hidden=256, eps=1e-6, residual_type=L.MOE_TYPE_BF16, weight_type=L.MOE_TYPE_BF16, x=4096, x_stride=256,
            residual=8192, residual_stride=256, weight=4096, num_tokens=2, codes=4096, scales=4096, y_bf16=0,
            residual_out=8192, residual_out_stride=256)


@pytest.mark.parametrize("kw,status", [
    (dict(hidden=0), L.MOE_ERR_INVALID_ARG),
    (dict(hidden=-128), L.MOE_ERR_INVALID_ARG),
    (dict(hidden=200), L.MOE_ERR_UNSUPPORTED),
    (dict(hidden=16512), L.MOE_ERR_UNSUPPORTED),
    (dict(eps=-1e-6), L.MOE_ERR_INVALID_ARG),
    (dict(eps=float("nan")), L.MOE_ERR_INVALID_ARG),
    (dict(eps=float("inf")), L.MOE_ERR_INVALID_ARG),
    (dict(residual_type=2), L.MOE_ERR_INVALID_ARG),
    (dict(weight_type=-1), L.MOE_ERR_INVALID_ARG),
    (dict(num_tokens=-1), L.MOE_ERR_INVALID_ARG),
    (dict(codes=0), L.MOE_ERR_INVALID_ARG),
    (dict(scales=0), L.MOE_ERR_INVALID_ARG),
    (dict(codes=0, scales=0), L.MOE_ERR_INVALID_ARG),
    (dict(residual=0), L.MOE_ERR_INVALID_ARG),
    (dict(x=0), L.MOE_ERR_INVALID_ARG),
    (dict(weight=0), L.MOE_ERR_INVALID_ARG),
    (dict(x=4104), L.MOE_ERR_INVALID_ARG),
    (dict(codes=4100), L.MOE_ERR_INVALID_ARG),
    (dict(scales=4098), L.MOE_ERR_INVALID_ARG),
    (dict(x_stride=128), L.MOE_ERR_INVALID_ARG),
    (dict(x_stride=260), L.MOE_ERR_INVALID_ARG),
    (dict(residual_stride=0), L.MOE_ERR_INVALID_ARG),
    (dict(residual_out_stride=-256), L.MOE_ERR_INVALID_ARG),
])
def test_bad_calls_are_refused(kw, status):
    with pytest.raises(L.MoEError) as ei:
        L.moe_rms_norm_quant(**{**GOOD, **kw})
    assert ei.value.status == status
    assert L.moe_last_error()


def test_no_tokens_is_no_launch():
    L.moe_rms_norm_quant(**{**GOOD, "num_tokens": 0})
    L.moe_rms_norm_quant(**{**GOOD, "num_tokens": 0, "x": 0, "residual": 0, "residual_out": 0})
