"""moe_rms_norm_quant in place: an output over its input takes the input's
rows (no GPU: the other strides are refused before a launch)."""

import pytest

from mixture_experts_ffn_route_amd import _lib as L
from tests.test_norm_host import GOOD


@pytest.mark.parametrize("kw,what", [
    (dict(residual_stride=512), "residual_out over residual"),
    (dict(residual_out_stride=512), "residual_out over residual"),
    (dict(x=16384, y_bf16=16384, x_stride=512), "y over x"),
])
def test_other_strides_are_refused(kw, what):
    with pytest.raises(L.MoEError, match=what) as ei:
        L.moe_rms_norm_quant(**{**GOOD, **kw})
    assert ei.value.status == L.MOE_ERR_INVALID_ARG
