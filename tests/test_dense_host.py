"""Host-side refusals of the dense products and the gated feed-forward block
(no GPU: every bad call returns before a launch), and the gradient's formula
against differences."""

import pytest
import torch

import mixture_experts_ffn_route_amd as m
from mixture_experts_ffn_route_amd import _lib as L
from tests import dense_util as D

KB, INVALID, UNSUPPORTED = 1 << 10, L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED

MATMUL = dict(x=1 << 20, x_stride=256, x_scale=2 << 20, w=3 << 20, w_stride=256, w_scale=4 << 20, m=3, n=200, k=256,
              add=5 << 20, add_stride=200, out=6 << 20, out_stride=200, workspace=0, ws_bytes=0)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(k=-16), INVALID),
    (dict(k=200), UNSUPPORTED), (dict(k=65552), UNSUPPORTED), (dict(n=262145), UNSUPPORTED),
    (dict(x=0), INVALID), (dict(w=0), INVALID), (dict(out=0), INVALID), (dict(x_scale=0), INVALID),
    (dict(w_scale=0), INVALID), (dict(x=(1 << 20) + 8), INVALID), (dict(w=(3 << 20) + 1), INVALID),
    (dict(x_scale=(2 << 20) + 2), INVALID), (dict(out=(6 << 20) + 1), INVALID), (dict(add=(5 << 20) + 1), INVALID),
    (dict(x_stride=240), INVALID), (dict(x_stride=264), INVALID), (dict(w_stride=0), INVALID),
    (dict(w_stride=1 << 22), INVALID), (dict(out_stride=199), INVALID), (dict(add_stride=0), INVALID),
    (dict(add=6 << 20, add_stride=208), INVALID),        # over out with another stride
    (dict(add=(6 << 20) + 200, add_stride=400, out_stride=400), INVALID),  # half over out's columns
    (dict(add=(6 << 20) + 400), INVALID),                # a row further
    (dict(out=(1 << 20) + 512), INVALID),                # over x
    (dict(out=(3 << 20) + 2), INVALID),                  # over w
    (dict(out=2 << 20), INVALID), (dict(out=4 << 20), INVALID),  # over the scales
])
def test_matmul_refusals(kw, status):
    with pytest.raises(L.MoEError) as e:
        L.moe_fp8_matmul(**{**MATMUL, **kw})
    assert e.value.status == status and L.moe_last_error()


def test_matmul_without_rows_launches_nothing():
    L.moe_fp8_matmul(**{**MATMUL, "m": 0, "x": 0, "out": 0, "add": 0})


def test_workspace_has_to_be_large_enough_and_aligned():
    m_, n, k = 300, 7168, 7168  # K in parts
    need = L.moe_fp8_matmul_workspace_query(m_, n, k)
    assert need > 0
    call = dict(MATMUL, m=m_, n=n, k=k, x_stride=k, w_stride=k, w=32 << 20, add=0, w_scale=128 << 20, x_scale=129 << 20,
                out=130 << 20, out_stride=n)
    for kw, status in ((dict(ws_bytes=need - 1, workspace=256 << 20), L.MOE_ERR_WORKSPACE_TOO_SMALL),
                       (dict(ws_bytes=need, workspace=0), INVALID),
                       (dict(ws_bytes=need, workspace=(256 << 20) + 16), INVALID)):
        with pytest.raises(L.MoEError) as e:
            L.moe_fp8_matmul(**{**call, **kw})
        assert e.value.status == status


FFN8 = dict(x=1 << 20, x_stride=256, x_scale=2 << 20, w13=3 << 20, w13_scale=4 << 20, w2=5 << 20, w2_scale=6 << 20,
            num_tokens=3, hidden=256, intermediate=128, add=0, add_stride=0, out=7 << 20, out_stride=256,
            workspace=8 << 20, ws_bytes=1 << 20)


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), INVALID), (dict(hidden=0), INVALID), (dict(intermediate=-128), INVALID),
    (dict(hidden=192), UNSUPPORTED), (dict(intermediate=64), UNSUPPORTED), (dict(hidden=65664), UNSUPPORTED),
    (dict(x=0), INVALID), (dict(w13=0), INVALID), (dict(w2=0), INVALID), (dict(x_scale=0), INVALID),
    (dict(w13_scale=0), INVALID), (dict(w2_scale=0), INVALID), (dict(out=0), INVALID),
    (dict(w13=(3 << 20) + 4), INVALID), (dict(w2=(5 << 20) + 8), INVALID), (dict(x_stride=128), INVALID),
    (dict(out_stride=255), INVALID), (dict(out=1 << 20), INVALID), (dict(out=3 << 20), INVALID),
    (dict(out=(5 << 20) - 2), INVALID), (dict(ws_bytes=0), L.MOE_ERR_WORKSPACE_TOO_SMALL), (dict(workspace=0), INVALID),
])
def test_shared_expert_refusals(kw, status):
    with pytest.raises(L.MoEError) as e:
        L.moe_ffn_fp8(**{**FFN8, **kw})
    assert e.value.status == status and L.moe_last_error()


FWD = dict(x=1 << 20, x_stride=64, w13=2 << 20, w2=3 << 20, num_tokens=3, hidden=64, intermediate=40, gate_up=4 << 20,
           h=5 << 20, out=6 << 20, out_stride=64, workspace=0, ws_bytes=0)


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), INVALID), (dict(hidden=0), INVALID), (dict(hidden=60), UNSUPPORTED),
    (dict(intermediate=44), UNSUPPORTED), (dict(intermediate=65544), UNSUPPORTED),
    (dict(x=0), INVALID), (dict(w13=0), INVALID), (dict(w2=0), INVALID), (dict(h=0), INVALID), (dict(out=0), INVALID),
    (dict(x=(1 << 20) + 2), INVALID), (dict(gate_up=(4 << 20) + 8), INVALID), (dict(x_stride=60), INVALID),
    (dict(x_stride=68), INVALID), (dict(out_stride=56), INVALID), (dict(x_stride=1 << 21), INVALID),
    (dict(out=1 << 20), INVALID), (dict(h=4 << 20), INVALID), (dict(gate_up=2 << 20), INVALID),
])
def test_forward_refusals(kw, status):
    with pytest.raises(L.MoEError) as e:
        L.moe_ffn_forward(**{**FWD, **kw})
    assert e.value.status == status and L.moe_last_error()


BWD = dict(dy=1 << 20, dy_stride=64, x=2 << 20, x_stride=64, w13=3 << 20, w2=4 << 20, gate_up=5 << 20, h=6 << 20,
           num_tokens=3, hidden=64, intermediate=40, dx=7 << 20, dx_stride=64, dw13=8 << 20, dw2=9 << 20, dw_type=0,
           accumulate=0, workspace=10 << 20, ws_bytes=1 << 20)


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), INVALID), (dict(hidden=60), UNSUPPORTED), (dict(dw_type=2), INVALID),
    (dict(accumulate=2), INVALID), (dict(accumulate=1), UNSUPPORTED), (dict(dy=0), INVALID), (dict(x=0), INVALID),
    (dict(w13=0), INVALID), (dict(w2=0), INVALID), (dict(gate_up=0), INVALID), (dict(h=0), INVALID),
    (dict(dw13=(8 << 20) + 8), INVALID), (dict(dy_stride=32), INVALID), (dict(dx_stride=68), INVALID),
    (dict(dx=1 << 20), INVALID), (dict(dw2=8 << 20), INVALID), (dict(dw13=2 << 20), INVALID),
    (dict(ws_bytes=16), L.MOE_ERR_WORKSPACE_TOO_SMALL), (dict(workspace=0), INVALID),
])
def test_backward_refusals(kw, status):
    with pytest.raises(L.MoEError) as e:
        L.moe_ffn_backward(**{**BWD, **kw})
    assert e.value.status == status and L.moe_last_error()


def test_wrappers_refuse_host_tensors():
    x, xs, w, ws = D.fp8_inputs(2, 128, 128, 0, device="cpu")
    with pytest.raises(ValueError, match="device"):
        m.fp8_matmul(x, xs, w, ws)
    with pytest.raises(ValueError, match="device"):
        m.MoESharedExpert(w, ws, w, ws)
    a, w13, w2, _ = D.ffn_inputs(2, 16, 8, 0, device="cpu")
    with pytest.raises(ValueError, match="device"):
        m.gated_ffn(a, w13, w2)


def test_gradient_formula_against_differences():
    t, h, i = 5, 16, 8
    x, w13, w2, dy = D.ffn_inputs(t, h, i, 3, device="cpu")
    want = D.ffn64(x, w13, w2, dy)
    base = [v.double() for v in (x, w13, w2)]

    def loss(*p):
        g, u = (p[0] @ p[1].T).split(i, 1)
        return ((g / (1 + torch.exp(-g)) * u) @ p[2].T * dy.double()).sum()

    gen = torch.Generator().manual_seed(1)
    for k, name in enumerate(("dx", "dw13", "dw2")):
        step = torch.randn(base[k].shape, generator=gen, dtype=torch.float64)
        plus, minus = list(base), list(base)
        plus[k], minus[k] = base[k] + 1e-5 * step, base[k] - 1e-5 * step
        difference = (loss(*plus) - loss(*minus)) / 2e-5
        assert abs((want[name][0] * step).sum() - difference) <= 1e-7 * (1 + abs(difference))


def test_bounds_reject_a_dropped_block():
    """A K-block left out of the 64-bit form lies beyond the bounds."""
    x, xs, w, ws = D.fp8_inputs(70, 128, 512, 0, device="cpu")
    want, bound = D.rounded(*D.product64(x, xs, w, ws))
    short = D.product64(x[:, :384].contiguous(), xs[:, :3], w[:, :384].contiguous(), ws[:, :3])[0]
    with pytest.raises(AssertionError):
        D.assert_within(short, want, bound, "short")
