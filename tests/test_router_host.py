"""Host-side refusals of the router's entry points (no GPU: every bad call
returns before a launch)."""

import pytest

from mixture_experts_ffn_route_amd import _lib as L


def _cfg(**kw):
    c = dict(hidden=7168, num_experts=256, top_k=8, score=L.MOE_SCORE_SIGMOID, num_groups=8, top_groups=4,
             renormalize=1, scale=2.5, expert_base=0, local_experts=256)
    c.update(kw)
    return L.moe_router_config_t(*c.values())


@pytest.mark.parametrize("kw,status", [
    (dict(hidden=0), L.MOE_ERR_INVALID_ARG),
    (dict(hidden=200), L.MOE_ERR_UNSUPPORTED),
    (dict(hidden=16512), L.MOE_ERR_UNSUPPORTED),
    (dict(num_experts=0), L.MOE_ERR_UNSUPPORTED),
    (dict(num_experts=1032), L.MOE_ERR_UNSUPPORTED),
    (dict(top_k=0), L.MOE_ERR_UNSUPPORTED),
    (dict(top_k=9), L.MOE_ERR_UNSUPPORTED),
    (dict(num_experts=4, num_groups=1, top_groups=1, local_experts=4), L.MOE_ERR_INVALID_ARG),
    (dict(score=2), L.MOE_ERR_INVALID_ARG),
    (dict(num_groups=0), L.MOE_ERR_UNSUPPORTED),
    (dict(num_groups=32), L.MOE_ERR_UNSUPPORTED),
    (dict(num_groups=7), L.MOE_ERR_INVALID_ARG),
    (dict(top_groups=0), L.MOE_ERR_INVALID_ARG),
    (dict(top_groups=9), L.MOE_ERR_INVALID_ARG),
    (dict(num_experts=32, num_groups=16, top_groups=2, local_experts=32), L.MOE_ERR_INVALID_ARG),  # 4 experts, K = 8
    (dict(num_experts=1000, num_groups=10, top_groups=4, local_experts=1000), L.MOE_ERR_UNSUPPORTED),  # 100 a lane
    (dict(renormalize=2), L.MOE_ERR_INVALID_ARG),
    (dict(scale=float("nan")), L.MOE_ERR_INVALID_ARG),
    (dict(expert_base=-1), L.MOE_ERR_INVALID_ARG),
    (dict(expert_base=1), L.MOE_ERR_INVALID_ARG),
    (dict(local_experts=0), L.MOE_ERR_INVALID_ARG),
    (dict(expert_base=2 ** 31 - 1, local_experts=256), L.MOE_ERR_INVALID_ARG),
])
def test_query_refuses_bad_configs(kw, status):
    with pytest.raises(L.MoEError) as ei:
        L.moe_router_workspace_query(_cfg(**kw), 64)
    assert ei.value.status == status
    assert L.moe_last_error()


@pytest.mark.parametrize("rows,status", [(0, L.MOE_ERR_INVALID_ARG), (-5, L.MOE_ERR_INVALID_ARG),
                                         ((1 << 24) + 1, L.MOE_ERR_UNSUPPORTED)])
def test_query_refuses_bad_sizes(rows, status):
    with pytest.raises(L.MoEError) as ei:
        L.moe_router_workspace_query(_cfg(), rows)
    assert ei.value.status == status


def test_workspace_grows_with_rows():
    sizes = [L.moe_router_workspace_query(_cfg(), r) for r in (1, 33, 1024, 1025, 8192, 8193, 32768, 1 << 20)]
    assert sizes == sorted(sizes) and all(s % 256 == 0 for s in sizes)
    assert sizes[0] >= 256 * 7168 * 2            # the weight fragments
    assert sizes[-1] >= (1 << 20) * 256 * 4      # one logit row per token


def test_create_refuses_before_any_launch():
    cfg = _cfg()
    n = L.moe_router_workspace_query(cfg, 64)
    for args, status in [
        ((0, 0, 4096, n), L.MOE_ERR_INVALID_ARG),              # no weight
        ((4104, 0, 4096, n), L.MOE_ERR_INVALID_ARG),           # misaligned weight
        ((4096, 4098, 4096, n), L.MOE_ERR_INVALID_ARG),        # misaligned bias
        ((4096, 4096, 0, n), L.MOE_ERR_INVALID_ARG),           # no workspace
        ((4096, 4096, 4112, n), L.MOE_ERR_INVALID_ARG),        # misaligned workspace
        ((4096, 4096, 4096, n - 1), L.MOE_ERR_WORKSPACE_TOO_SMALL),
    ]:
        with pytest.raises(L.MoEError) as ei:
            L.moe_router_create(cfg, 64, *args)
        assert ei.value.status == status
    with pytest.raises(L.MoEError) as ei:  # a bias would reorder softmax scores
        L.moe_router_create(_cfg(score=L.MOE_SCORE_SOFTMAX), 64, 4096, 4096, 4096, 1 << 30)
    assert ei.value.status == L.MOE_ERR_UNSUPPORTED


def test_null_handle():
    with pytest.raises(L.MoEError) as ei:
        L.moe_router_forward(0, 4096, 7168, 1, 4096, 4096)
    assert ei.value.status == L.MOE_ERR_INVALID_ARG
    L.moe_router_destroy(0)
