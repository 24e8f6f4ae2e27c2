"""Every form that the dense products take (kernel, tile, width, parts of K, cut
last K-block, epilogue), against 64-bit arithmetic.  test_dense_plans.py checks
that these sizes, with those of test_gpu_linear.py and test_gpu_ffn.py, reach
them all."""

import pytest
import torch

from tests import dense_plans as P
from tests import dense_util as D

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_route_amd as pkg
    return pkg


PRODUCTS = [
    # few rows: 1 to 4 blocks of 16 a workgroup, 16 and 32 columns
    (9, 7208, 528), (18, 4320, 512), (20, 5049, 528), (35, 2264, 512), (36, 2179, 560), (65, 2066, 512), (34, 4208, 544),
    (50, 2168, 512), (50, 2336, 528), (2712, 73, 512),
    # 128 x 128 tiles
    (76, 13400, 544), (690, 65, 15104), (420, 1262, 5360), (11712, 559, 512), (6597, 1032, 576), (300, 7168, 7168),
    (17, 8408, 4320), (33, 1589, 12208),
    # 128 x 256
    (269, 12008, 544), (18, 9442, 3712), (20, 9587, 4784), (2505, 715, 13808),
    # 256 x 256
    (4096, 7168, 2048), (523, 13800, 512), (1921, 4216, 528), (1859, 13084, 256), (513, 14579, 560), (134, 11616, 4480),
    (11390, 137, 4912),
]


@pytest.mark.parametrize("rows,n,k", PRODUCTS)
@pytest.mark.parametrize("with_add", [False, True])
def test_product(m, rows, n, k, with_add):
    x, xs, w, ws = D.fp8_inputs(rows, n, k, rows * 3 + n)
    add = torch.randn(rows, n, device="cuda").bfloat16() if with_add else None
    want, bound = D.rounded(*D.product64(x, xs, w, ws), add)
    D.assert_within(m.fp8_matmul(x, xs, w, ws, add=add), want, bound, P.product_fp8(rows, n, k)[0])


# a row stride of out and add that leaves 2, 8 or 16 bytes to be stored at once
STRIDED = [(rows, n, k, pad) for rows, n, k in [(300, 1280, 7168), (2505, 712, 5000 - 8), (1859, 3400, 256), (134, 11616, 4480)]
           for pad in (9, 12, 16)]


@pytest.mark.parametrize("rows,n,k,pad", STRIDED)
def test_strided_rows_and_output_over_add(m, rows, n, k, pad):
    x, xs, w, ws = D.fp8_inputs(rows, n, k, rows + pad)
    xw = torch.full((rows, k + 48), 0x7F, dtype=torch.uint8, device="cuda")
    xw[:, 32:32 + k] = x
    wide = torch.randn(rows + 1, n + pad, device="cuda").bfloat16()
    at = pad - 8  # columns in front: 2, 8 or 16 bytes
    left = wide.clone()
    view = wide[:rows, at:at + n]
    want, bound = D.rounded(*D.product64(x, xs, w, ws), view)
    got = m.fp8_matmul(xw[:, 32:32 + k], xs, w, ws, add=view, out=view)
    assert got.data_ptr() == view.data_ptr()
    D.assert_within(got, want, bound, P.product_fp8(rows, n, k, pad == 16)[0])
    left[:rows, at:at + n] = view
    assert torch.equal(left, wide)  # nothing beside the rows was written


SHARED = [(18, 512, 2176), (18, 5888, 512), (66, 4224, 3328), (66, 7168, 4352), (136, 1408, 768), (193, 896, 512),
          (198, 6272, 512), (256, 7168, 2048), (397, 5376, 4480), (397, 5504, 7552), (1034, 7296, 512), (10948, 640, 512),
          (4096, 7168, 2048)]


@pytest.mark.parametrize("t,h,i", SHARED)
@pytest.mark.parametrize("with_add", [False, True])
def test_shared_expert(m, t, h, i, with_add):
    x, xs, w13, s13 = D.fp8_inputs(t, 2 * i, h, t + h)
    _, _, w2, s2 = D.fp8_inputs(1, h, i, t + i)
    add = torch.randn(t, h, device="cuda").bfloat16() if with_add else None
    want, bound = D.shared64(x, xs, w13, s13, w2, s2, add)
    got = m.MoESharedExpert(w13, s13, w2, s2).forward(x, xs, add=add)
    D.assert_within(got, want, bound, str(P.shared_expert(t, h, i)))
    # half a step of out and of a neighbouring code of h, as in test_gpu_linear.py
    assert D.rel_rms(got, want) < 2 * D.HALF_BF16 / 3 ** 0.5


FFN = [(1, 3136, 5072), (1, 6608, 1120), (1, 1104, 7136), (1, 1152, 6248), (2, 5456, 7680), (19, 6208, 2496),
       (20, 5008, 3112), (34, 5824, 4608), (64, 2112, 1856), (64, 2440, 4392), (64, 3200, 5440), (64, 3656, 1072),
       (64, 5568, 1344), (72, 2280, 1040), (74, 2112, 1728), (129, 952, 272), (161, 6312, 6072), (262, 4840, 3344),
       (268, 256, 272), (268, 464, 256), (320, 4992, 1600), (641, 3536, 5920), (704, 5504, 3200), (891, 1560, 4976),
       (1042, 3968, 3720), (2125, 4808, 272), (5516, 320, 1912), (5789, 312, 4608), (6168, 3016, 1320), (7472, 1096, 256),
       (11200, 288, 320), (11328, 568, 256), (11904, 256, 576), (12382, 576, 264), (4096, 7168, 2048)]


@pytest.mark.parametrize("t,h,i", FFN)
def test_block_and_gradients(m, t, h, i):
    x, w13, w2, dy = D.ffn_inputs(t, h, i, t + h + i)
    want = D.ffn64(x, w13, w2, dy)
    alone = m.gated_ffn(x, w13, w2)
    leaves = [v.requires_grad_(True) for v in (x, w13, w2)]
    y = m.gated_ffn(*leaves)
    got = dict(zip(("dx", "dw13", "dw2"), torch.autograd.grad(y, leaves, dy)), y=y.detach())
    assert torch.equal(alone, got["y"])
    forms = P.ffn_forward(t, h, i)[0] + P.ffn_backward(t, h, i)[0]
    half = D.HALF_BF16 / 3 ** 0.5
    for name, g in got.items():
        value, bound = want[name] if name in ("y", "dx") else D.rounded(*want[name])
        D.assert_within(g, value, bound, f"{name} {forms}")
        # two roundings count, as in test_gpu_ffn.py
        assert D.rel_rms(g, value) < 2 ** 0.5 * half, name


FLOAT32 = [(256, 136, 128), (277, 144, 128), (256, 520, 6736), (256, 7256, 1040), (270, 6904, 528), (265, 5784, 1392),
           (269, 1352, 5912), (320, 4960, 1608), (4096, 7168, 2048)]


@pytest.mark.parametrize("t,h,i", FLOAT32)
def test_float32_weight_gradients_and_accumulation(m, t, h, i):
    x, w13, w2, dy = D.ffn_inputs(t, h, i, t + i)
    want = D.ffn64(x, w13, w2, dy)
    forms = P.ffn_backward(t, h, i, True)[0][2:]
    _, gu, hid = m.gated_ffn_forward(x, w13, w2)
    dw13, dw2 = torch.full((2 * i, h), float("nan"), device="cuda"), torch.full((h, i), float("nan"), device="cuda")
    m.gated_ffn_backward(dy, x, w13, w2, gu, hid, dw13=dw13, dw2=dw2)
    D.assert_within(dw13, *want["dw13"], f"dw13 {forms}")
    D.assert_within(dw2, *want["dw2"], f"dw2 {forms}")
    b13, b2 = torch.randn_like(dw13), torch.randn_like(dw2)
    a13, a2 = b13.clone(), b2.clone()
    m.gated_ffn_backward(dy, x, w13, w2, gu, hid, dw13=a13, dw2=a2, accumulate=True)
    assert torch.equal(a13, b13 + dw13) and torch.equal(a2, b2 + dw2)


# ---------------------------------------------------------------------------
# Parts of K: calls beside each other and replays have workspaces of their own
# ---------------------------------------------------------------------------

PARTS = [(300, 7168, 7168), (420, 1262, 5360), (2505, 715, 13808), (134, 11616, 4480)]


def _parts_calls(m, rows, n, k):
    """A product, a shared expert and a BF16 block whose K is in parts."""
    x, xs, w, ws = D.fp8_inputs(rows, n, k, 1)
    a, sa, w13, s13 = D.fp8_inputs(256, 2 * 2048, 7168, 2)
    _, _, w2, s2 = D.fp8_inputs(1, 7168, 2048, 3)
    b, v13, v2, dy = D.ffn_inputs(256, 7168, 2048, 4)
    shared = m.MoESharedExpert(w13, s13, w2, s2)
    grads = [torch.empty_like(v) for v in (b, v13, v2)]

    def block():
        y, gu, h = m.gated_ffn_forward(b, v13, v2)
        out = [torch.empty_like(g) for g in grads]
        m.gated_ffn_backward(dy, b, v13, v2, gu, h, dx=out[0], dw13=out[1], dw2=out[2])
        return [y, *out]

    from mixture_experts_ffn_route_amd import _lib as L
    assert L.moe_fp8_matmul_workspace_query(rows, n, k) > 0 and L.moe_ffn_workspace_query(256, 7168, 2048)[0] > 0
    assert "parts" in P.shared_expert(256, 7168, 2048)[0] and "parts" in P.ffn_backward(256, 7168, 2048)[0][0]
    return (x, xs, a, sa, b), lambda: [m.fp8_matmul(x, xs, w, ws), shared.forward(a, sa), *block()]


@pytest.mark.parametrize("rows,n,k", PARTS)
def test_repeats_and_two_streams_give_the_same_bits(m, rows, n, k):
    _, call = _parts_calls(m, rows, n, k)
    want = call()
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(call())
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(g, w) for g, w in zip(out, want))


@pytest.mark.parametrize("rows,n,k", PARTS[:2])
def test_two_graphs_replayed(m, rows, n, k):
    inputs, call = _parts_calls(m, rows, n, k)
    call()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = call()
        graphs.append((g, outs))
    for seed in range(3):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for v in (inputs[0], inputs[2]):
            v.copy_(torch.randint(0, 120, v.shape, generator=gen, device="cuda", dtype=torch.uint8))
        inputs[4].copy_(torch.randn(inputs[4].shape, generator=gen, device="cuda"))
        want = call()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
            for v in outs:
                v.zero_()


@pytest.mark.parametrize("rows,n,k", [(300, 2560, 7168), (2505, 715, 5000 - 8), (1859, 2600, 400), (4096, 4224, 640)])
def test_nan_stays_in_its_row_and_column(m, rows, n, k):
    x, xs, w, ws = D.fp8_inputs(rows, n, k, 12)
    plain = m.fp8_matmul(x, xs, w, ws)
    x[1, k - 1] = 0x7F
    xs[rows - 1, 1] = float("nan")
    w[200, 3] = 0xFF
    got = m.fp8_matmul(x, xs, w, ws)
    bad = torch.zeros(rows, n, dtype=torch.bool, device="cuda")
    bad[1], bad[rows - 1], bad[:, 200] = True, True, True
    assert torch.equal(got.isnan(), bad)
    assert torch.equal(got[~bad], plain[~bad])
