"""MoELayer and MoEBlock launch on the layer's device, whatever the current
one is (no GPU: the library's calls are recorded)."""

import contextlib
import types

import pytest
import torch

from mixture_experts_ffn_route_amd import MoEBlock, MoELayer, block as block_module, layer as layer_module


@pytest.fixture
def record(monkeypatch):
    """Device 0 is current; the layer lives on device 1."""
    state = types.SimpleNamespace(current=0, calls=[])

    @contextlib.contextmanager
    def device(d):
        before, state.current = state.current, torch.device(d).index
        yield
        state.current = before

    def called(name):
        return lambda *args: state.calls.append((name, state.current, args[-1]))

    monkeypatch.setattr(torch.cuda, "current_device", lambda: state.current)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda *a: types.SimpleNamespace(cuda_stream=1000 + state.current))
    monkeypatch.setattr(layer_module, "current_raw_stream", lambda index: 1000 + index)
    for name in ("moe_stage_inputs", "moe_layer_forward", "moe_layer_forward_noalloc", "moe_read_status"):
        monkeypatch.setattr(layer_module.L, name, called(name))
    return state


def _layer():
    layer = object.__new__(MoELayer)
    layer.hidden, layer.top_k, layer.max_rows, layer.handle = 128, 2, 32, None
    layer.workspace = types.SimpleNamespace(device=torch.device("cuda", 1))
    layer.capacity_factor = 1.0
    layer.cfg = types.SimpleNamespace(num_experts=4, act_format=block_module.L.MOE_ACT_E4M3_1X128)
    return layer


def test_every_call_runs_on_the_layers_device(record):
    layer = _layer()
    x, out = torch.zeros(3, 128).bfloat16(), torch.zeros(3, 128).bfloat16()
    idx, w = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    layer.stage(x, idx, w, out=out)
    layer.forward()
    layer.forward_noalloc(x, idx, w, out)
    layer.status()
    assert [c[0] for c in record.calls] == ["moe_stage_inputs", "moe_layer_forward", "moe_layer_forward_noalloc",
                                            "moe_read_status"]
    assert all(c[1:] == (1, 1001) for c in record.calls if c[0] != "moe_layer_forward_noalloc")
    assert all(c[1] == 1 for c in record.calls) and record.current == 0
    record.calls.clear()
    record.current = 1   # the layer's device is current already
    layer.forward()
    assert record.calls == [("moe_layer_forward", 1, 1001)]


def test_block_refuses_a_router_on_another_device():
    router = types.SimpleNamespace(hidden=128, top_k=2, device=torch.device("cuda", 0),
                                   cfg=types.SimpleNamespace(local_experts=4))
    with pytest.raises(ValueError, match="device"):
        MoEBlock(None, router, _layer())


@pytest.mark.parametrize("fp8,hidden,top_k,experts,here,few", [
    (True, 7168, 8, 32, 32, 6), (True, 2048, 6, 32, 32, 8), (True, 7168, 8, 256, 32, 16), (True, 128, 1, 4, 4, 16),
    (True, 7296, 4, 16, 16, 4), (True, 10368, 4, 16, 16, 2), (True, 16384, 8, 256, 32, 8),
    (False, 7168, 8, 32, 32, 5), (False, 16384, 8, 256, 32, 12), (False, 2048, 8, 64, 32, 10)])
def test_few_token_limit_goes_by_the_routes_expected_here(fp8, hidden, top_k, experts, here, few):
    layer = _layer()
    layer.hidden = hidden
    layer.top_k, layer.cfg.num_experts = top_k, here
    layer.cfg.act_format = block_module.L.MOE_ACT_E4M3_1X128 if fp8 else block_module.L.MOE_ACT_BF16
    router = types.SimpleNamespace(hidden=hidden, top_k=top_k, device=layer.workspace.device,
                                   cfg=types.SimpleNamespace(local_experts=here, num_experts=experts, top_k=top_k))
    assert MoEBlock(None, router, layer).few == few
    layer.capacity_factor = 0.5
    assert MoEBlock(None, router, layer).few == 0
