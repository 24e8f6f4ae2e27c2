"""Workspaces that a caller supplies: what lies between a view's elements is
not the handle's."""

import pytest
import torch

from synthetic import MoEShape, make_layer_inputs
from tests.test_gpu_router import _inputs, check, reference

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_ffn_route_amd import MoELayer, MoERouter
    from mixture_experts_ffn_route_amd.harness import to_device


def test_router_workspace():
    x, w, _ = _inputs(8, 256, 40, 1)
    n = MoERouter(w, 4, max_rows=8).ws_bytes
    whole = torch.empty(2 * n, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        MoERouter(w, 4, max_rows=8, workspace=whole[::2])
    r = MoERouter(w, 4, max_rows=8, workspace=whole)
    check(r, x, reference(x, w, 4, "softmax"), experts=40)


def test_layer_workspace():
    dev = to_device(make_layer_inputs(MoEShape(4, 256, 128, 4, 2, "topk"), seed=1))
    args = (256, 128, 4, 2, dev.w13, dev.w13_scale, dev.w2, dev.w2_scale)
    n = MoELayer(*args, expected_m=2, max_rows=4).ws_bytes
    whole = torch.empty(2 * n, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        MoELayer(*args, expected_m=2, max_rows=4, workspace=whole[::2])
    MoELayer(*args, expected_m=2, max_rows=4, workspace=whole)
