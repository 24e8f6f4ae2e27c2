"""The e4m3 matrix product with block scales and the shared expert, against
64-bit arithmetic."""

import pytest
import torch

from tests import dense_util as D

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_route_amd as pkg
    return pkg


SIZES = [(1, 1, 16), (1, 7168, 2048), (5, 130, 144), (16, 1003, 2000), (17, 64, 128), (33, 257, 1040), (64, 512, 4096),
         (65, 1, 16), (65, 130, 144), (100, 1003, 2000), (128, 128, 128), (129, 640, 7168), (300, 257, 400),
         (513, 1027, 2064), (1100, 2304, 640),
         (2500, 2500, 400), (2341, 2563, 1040), (3000, 2304, 128), (4100, 1541, 256)]


@pytest.mark.parametrize("rows,n,k", SIZES)
@pytest.mark.parametrize("with_add", [False, True])
def test_product(m, rows, n, k, with_add):
    x, xs, w, ws = D.fp8_inputs(rows, n, k, rows * 7 + n)
    add = torch.randn(rows, n, device="cuda").bfloat16() if with_add else None
    got = m.fp8_matmul(x, xs, w, ws, add=add)
    want, bound = D.rounded(*D.product64(x, xs, w, ws), add)
    D.assert_within(got, want, bound, f"{rows}x{n}x{k}")


@pytest.mark.parametrize("rows", [3, 40, 200, 13000])
def test_strided_rows_and_output_over_add(m, rows):
    n, k = 260, 272
    x, xs, w, ws = D.fp8_inputs(rows, n, k, rows)
    xw = torch.full((rows, k + 48), 0x7F, dtype=torch.uint8, device="cuda")
    xw[:, 16:16 + k] = x
    ww = torch.full((n, k + 16), 0x7F, dtype=torch.uint8, device="cuda")
    ww[:, :k] = w
    wide = torch.randn(rows + 1, n + 9, device="cuda").bfloat16()
    before = wide.clone()
    add = wide[:rows, 3:3 + n]  # not even 8-byte aligned
    want, bound = D.rounded(*D.product64(x, xs, w, ws), add)
    got = m.fp8_matmul(xw[:, 16:16 + k], xs, ww[:, :k], ws, add=add, out=add)
    assert got.data_ptr() == add.data_ptr()
    D.assert_within(got, want, bound, "strided")
    left = before.clone()
    left[:rows, 3:3 + n] = wide[:rows, 3:3 + n]
    assert torch.equal(left, wide)  # nothing beside the rows was written


@pytest.mark.parametrize("rows", [2, 30, 150, 13000])
def test_scales_of_far_apart_blocks(m, rows):
    n, k = 300, 1024
    x, xs, w, ws = D.fp8_inputs(rows, n, k, 11)
    gen = torch.Generator(device="cuda").manual_seed(5)
    xs = xs * torch.exp2(torch.randint(-40, 20, xs.shape, generator=gen, device="cuda").float())
    xs[0] = 0.0  # a row of zero scales
    want, bound = D.rounded(*D.product64(x, xs, w, ws))
    got = m.fp8_matmul(x, xs, w, ws)
    D.assert_within(got, want, bound, "far scales")
    assert not got[0].any()


@pytest.mark.parametrize("rows", [3, 40, 130, 700, 13000])
def test_nan_stays_in_its_row_and_column(m, rows):
    n, k = 384, 400
    x, xs, w, ws = D.fp8_inputs(rows, n, k, 12)
    plain = m.fp8_matmul(x, xs, w, ws)
    x[1, 399] = 0x7F
    xs[2, 1] = float("nan")
    w[200, 3] = 0xFF
    got = m.fp8_matmul(x, xs, w, ws)
    bad = torch.zeros(rows, n, dtype=torch.bool, device="cuda")
    bad[1], bad[2], bad[:, 200] = True, True, True
    assert torch.equal(got.isnan(), bad)
    assert torch.equal(got[~bad], plain[~bad])


@pytest.mark.parametrize("rows", [1, 64, 65, 600])
def test_zero_and_subnormal_codes(m, rows):
    n, k = 160, 256
    x = torch.randint(0, 8, (rows, k), dtype=torch.uint8, device="cuda")  # 0 and the subnormals
    w = torch.randint(0, 8, (n, k), dtype=torch.uint8, device="cuda") | 0x80
    xs, ws = torch.ones(rows, 2, device="cuda"), torch.ones(2, 2, device="cuda")
    want, bound = D.rounded(*D.product64(x, xs, w, ws))
    D.assert_within(m.fp8_matmul(x, xs, w, ws), want, bound, "subnormals")


def test_no_rows(m):
    x, xs, w, ws = D.fp8_inputs(1, 64, 128, 0)
    assert m.fp8_matmul(x[:0], xs[:0], w, ws).shape == (0, 64)


@pytest.mark.parametrize("rows,n,k", [(40, 512, 512), (90, 700, 2048), (520, 512, 256), (4096, 2048, 1024)])
def test_repeats_give_the_same_bits(m, rows, n, k):
    x, xs, w, ws = D.fp8_inputs(rows, n, k, 3)
    first = m.fp8_matmul(x, xs, w, ws)
    for _ in range(3):
        assert torch.equal(m.fp8_matmul(x, xs, w, ws), first)


SHARED = [(1, 256, 128), (1, 7168, 2048), (16, 1280, 640), (17, 512, 384), (48, 2048, 768), (64, 256, 128),
          (65, 256, 128), (77, 2048, 768), (301, 1152, 896), (1200, 512, 1024),
          (2341, 2560, 1280), (700, 7168, 8192 - 128)]


@pytest.mark.parametrize("t,h,i", SHARED)
@pytest.mark.parametrize("with_add", [False, True])
def test_shared_expert(m, t, h, i, with_add):
    x, xs, w13, s13 = D.fp8_inputs(t, 2 * i, h, t + h)
    _, _, w2, s2 = D.fp8_inputs(1, h, i, t + i)
    add = torch.randn(t, h, device="cuda").bfloat16() if with_add else None
    want, bound = D.shared64(x, xs, w13, s13, w2, s2, add)
    shared = m.MoESharedExpert(w13, s13, w2, s2)
    got = shared.forward(x, xs, add=add)
    D.assert_within(got, want, bound, f"{t}x{h}x{i}")
    # out and h's codes are rounded; a code that falls to its neighbour is rare:
    # errors of half a step each, 2^-8 / sqrt(3), and as much again for those
    assert D.rel_rms(got, want) < 2 * D.HALF_BF16 / 3 ** 0.5
    if add is not None:
        assert torch.equal(shared.forward(x, xs, add=add, out=add), got)


@pytest.mark.parametrize("t", [2, 30, 70, 1100, 12500])
def test_shared_expert_rows_that_are_not_finite(m, t):
    h, i = 512, 256
    x, xs, w13, s13 = D.fp8_inputs(t, 2 * i, h, 1)
    _, _, w2, s2 = D.fp8_inputs(1, h, i, 2)
    shared = m.MoESharedExpert(w13, s13, w2, s2)
    plain = shared.forward(x, xs)
    xs[0, 0] = float("nan")
    xs[1] = 0.0
    got = shared.forward(x, xs)
    assert got[0].isnan().all()
    assert not got[1].any()
    assert torch.equal(got[2:], plain[2:])


@pytest.mark.parametrize("t", [4, 20, 100])
def test_captured_and_replayed(m, t):
    h, i = 1024, 512
    x, xs, w13, s13 = D.fp8_inputs(t, 2 * i, h, 5)
    _, _, w2, s2 = D.fp8_inputs(1, h, i, 6)
    shared = m.MoESharedExpert(w13, s13, w2, s2)
    shared.forward(x, xs)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs of the same sizes
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = shared.forward(x, xs)
            z = m.fp8_matmul(x, xs, w13, s13)
        graphs.append((g, y, z))
    for seed in range(3):
        nx, ns, _, _ = D.fp8_inputs(t, 1, h, 100 + seed)
        x.copy_(nx)
        xs.copy_(ns)
        want, other = shared.forward(x, xs), m.fp8_matmul(x, xs, w13, s13)
        for g, y, z in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want) and torch.equal(z, other)


def test_two_streams_at_once(m):
    x, xs, w, ws = D.fp8_inputs(100, 600, 4096, 8)
    want = m.fp8_matmul(x, xs, w, ws)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(m.fp8_matmul(x, xs, w, ws))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_offsets_beyond_32_bits(m):
    """5 GB of rows: the last ones equal the same rows by themselves, which take
    the few-row form, within both forms' bounds."""
    rows, n, k = 300000, 64, 16384
    x = torch.randint(0, 120, (rows, k), dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    xs = torch.rand(rows, k // 128, generator=gen, device="cuda")
    _, _, w, ws = D.fp8_inputs(1, n, k, 2)
    got = m.fp8_matmul(x, xs, w, ws)
    for at in (0, rows // 2, rows - 70):
        sl = slice(at, at + 70)
        want, bound = D.rounded(*D.product64(x[sl].contiguous(), xs[sl].contiguous(), w, ws))
        D.assert_within(got[sl], want, bound, f"rows from {at}")
