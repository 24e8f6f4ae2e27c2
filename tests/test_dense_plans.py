"""That the GPU tests of the dense products reach every form the library takes,
and that dense_plans.py takes the library's choice."""

import random

import pytest

from mixture_experts_ffn_route_amd import _lib as L
from tests import dense_plans as P
from tests import test_gpu_dense_forms as forms
from tests import test_gpu_ffn as ffn
from tests import test_gpu_linear as linear


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _product(rng):
    n, k = _log_int(rng, 1, 16384), 16 * _log_int(rng, 1, 1024)
    if rng.random() < 0.5:
        n = (n + 7) // 8 * 8
    if rng.random() < 0.5:
        k = (k + 127) // 128 * 128
    return _log_int(rng, 1, 16384), n, k


def _shared(rng):
    return _log_int(rng, 1, 32768), 128 * rng.randint(2, 64), 128 * _log_int(rng, 1, 64)


def _block(rng):
    size = [_log_int(rng, 1, 16384), 8 * rng.randint(32, 1024), 8 * _log_int(rng, 16, 1024)]
    return [(v + 63) // 64 * 64 if rng.random() < 0.4 else v for v in size]


def test_the_librarys_workspaces_are_those_of_the_same_plans():
    rng = random.Random(1)
    parts = 0
    for _ in range(3000):
        size = _product(rng)
        want = P.product_fp8(*size)[1]
        assert L.moe_fp8_matmul_workspace_query(*size) == want, size
        parts += want > 0
        size = _shared(rng)
        assert L.moe_ffn_fp8_workspace_query(*size) == P.shared_bytes(*size), size
        size = _block(rng)
        assert L.moe_ffn_workspace_query(*size) == (P.ffn_forward(*size)[1], P.ffn_backward(*size)[1]), size
    assert parts > 50


def _forms_of(op, size):
    if op == "product":
        return {P.product_fp8(*size)[0]}
    if op == "shared":
        pair = P.shared_expert(*size)
        return set() if pair is None else {f"{which}: {f}" for which, f in zip(("gate|up", "down"), pair)}
    if op == "float32":
        return {f"{which}: {f}" for which, f in zip(("dw13", "dw2"), P.ffn_backward(*size, True)[0][2:])}
    both = P.ffn_forward(*size)[0] + P.ffn_backward(*size)[0]
    return {f"{which}: {f}" for which, f in zip(("gate|up", "down", "dh", "dx", "dw13", "dw2"), both)}


TESTED = {"product": linear.SIZES + forms.PRODUCTS, "shared": linear.SHARED + forms.SHARED,
          "block": ffn.SIZES + forms.FFN, "float32": forms.FLOAT32}
RANDOM = {"product": _product, "shared": _shared, "block": _block, "float32": _block}
LARGEST = {"product": 16384 * 7168 * 7168, "shared": 32768 * 7168 * 2048, "block": 16384 * 7168 * 2048,
           "float32": 4096 * 7168 * 2048}


@pytest.mark.parametrize("op", list(TESTED))
def test_every_form_that_sizes_take_is_tested(op):
    tested = set().union(*(_forms_of(op, s) for s in TESTED[op]))
    rng = random.Random(2)
    missing = {}
    for _ in range(6000):
        size = RANDOM[op](rng)
        if size[0] * size[1] * size[2] <= LARGEST[op]:
            missing.update({f: size for f in _forms_of(op, size) - tested})
    assert not missing


def test_sizes_in_parts_have_parts():
    for size in forms.PARTS:
        assert "parts" in P.product_fp8(*size)[0] and L.moe_fp8_matmul_workspace_query(*size) > 0
