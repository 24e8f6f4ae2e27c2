"""moe_layer_decode: what it refuses before it looks at the device."""

import pytest

from mixture_experts_ffn_route_amd import _lib as L


def test_a_missing_layer_is_refused():
    with pytest.raises(L.MoEError, match="layer is NULL") as e:
        L.moe_layer_decode(0, 4096, 0, 4096, 4096, 1, 4096)
    assert e.value.status == L.MOE_ERR_INVALID_ARG


def test_the_workspace_holds_the_few_token_regions():
    """h in FP32 and e4m3 with its scales, the plan and a counter per block of
    h for each route of a call."""
    def query(max_rows):
        cfg = L.moe_config_t(256, 1024, 4, 2, L.MOE_WEIGHT_E4M3_BLOCK128, L.MOE_ACT_E4M3_1X128, 0)
        return L.moe_workspace_query(cfg, 1, max_rows, 1.0)

    routes, inter = 2, 1024
    per_token = routes * (inter * 5 + inter // 128 * 4 + inter // 128 * 4)
    # up to 16 tokens each one adds its routes
    assert query(16) - query(1) >= 15 * per_token
