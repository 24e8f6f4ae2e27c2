"""Where the router's ids are hardest to get right: selection biases of any
size, rows and gates whose logits lie close for a reason, sums that cancel.

Every choice is that of 64-bit arithmetic (``ids_64``): a NaN ranks below every
number, ties go to the lowest group and expert.
"""

import numpy as np
import pytest
import torch

from tests.test_gpu_router import U, _inputs

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_ffn_route_amd import MoERouter


def _descending(v):
    """Positions of ``v``'s rows in descending order; a NaN after -inf, ties by position."""
    return np.lexsort((-np.where(np.isnan(v), -np.inf, v), np.isnan(v)), axis=-1)


def ids_64(logits, score, K, bias=None, groups=1, top_groups=1):
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    with np.errstate(all="ignore"):
        choice = logits if score == "softmax" else 1.0 / (1.0 + np.exp(-logits))
        if bias is not None:
            choice = choice + bias.double().cpu().numpy()
        gone = np.zeros((T, E), dtype=bool)
        if top_groups < groups:
            n = E // groups
            by = choice.reshape(T, groups, n)
            top = np.take_along_axis(by, _descending(by), axis=2)
            value = top[:, :, 0] if score == "softmax" or n == 1 else top[:, :, 0] + top[:, :, 1]
            out = _descending(value)[:, top_groups:]
            for g in range(out.shape[1]):
                for j in range(n):
                    gone[np.arange(T), out[:, g] * n + j] = True
        # experts of other groups after everything else
        order = np.lexsort((-np.where(np.isnan(choice), -np.inf, choice), np.isnan(choice), gone), axis=-1)
    return order[:, :K]


def _logits(x, w):
    with np.errstate(all="ignore"):
        return x.double().cpu().numpy() @ w.double().cpu().numpy().T


def _ids(x, w, K, **kw):
    r = MoERouter(w, K, max_rows=x.shape[0], **kw)
    ids = torch.empty(x.shape[0], K, dtype=torch.int32, device="cuda")
    r.route(x, ids=ids)
    return ids.cpu().numpy()


def _close_gates(H, E, seed):
    """Gates that differ in the last places of a few elements: the logits of a
    row lie within about 1e-5 of each other."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn(1, H, generator=g, device="cuda") * H ** -0.5).bfloat16().expand(E, H).clone()
    w[:, :8] = (3e-6 * torch.randn(E, 8, generator=g, device="cuda")).bfloat16()
    return w


@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 4)])
@pytest.mark.parametrize("off", [-1e4, -1e9, -3e38, 1e9, float("-inf"), float("inf"), float("nan")])
def test_one_bias_of_any_size(off, groups, top_groups):
    T, H, E, K = 700, 512, 256, 8
    w = _close_gates(H, E, 3)
    x, _, _ = _inputs(T, H, 1, 3)
    bias = 1e-6 * torch.randn(E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    bias[37] = off
    got = _ids(x, w, K, score="sigmoid", bias=bias, num_groups=groups, top_groups=top_groups)
    assert np.array_equal(got, ids_64(_logits(x, w), "sigmoid", K, bias, groups, top_groups))


@pytest.mark.parametrize("E,groups,top_groups", [(64, 1, 1), (256, 8, 4), (256, 8, 7), (1024, 16, 5)])
@pytest.mark.parametrize("off", [-1e9, float("-inf"), float("nan")])
def test_most_experts_switched_off(E, groups, top_groups, off):
    """Whole groups of them, groups with one expert left, and fewer experts
    left than the token takes."""
    T, H, K = 90, 512, 8
    x, w, b = _inputs(T, H, E, 5, bias=True)
    g = torch.Generator().manual_seed(E)
    for left in (3, K, E // 4):
        bias = b.clone()
        bias[torch.randperm(E, generator=g)[left:].cuda()] = off
        got = _ids(x, w, K, score="sigmoid", bias=bias, num_groups=groups, top_groups=top_groups)
        want = ids_64(_logits(x, w), "sigmoid", K, bias, groups, top_groups)
        assert np.array_equal(got, want), left


@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 3)])
@pytest.mark.parametrize("common", [-3e4, 1e6, 1e9])
def test_large_common_biases(common, groups, top_groups):
    """All biases large: FP32 tells none of the choices apart, FP64 most."""
    T, H, E, K = 60, 512, 256, 8
    x, _, _ = _inputs(T, H, 1, 2)
    w = _close_gates(H, E, 2)
    bias = torch.full((E,), common, device="cuda")
    got = _ids(x, w, K, score="sigmoid", bias=bias, num_groups=groups, top_groups=top_groups)
    assert np.array_equal(got, ids_64(_logits(x, w), "sigmoid", K, bias, groups, top_groups))


@pytest.mark.parametrize("E", [40, 256, 640])
@pytest.mark.parametrize("step", [1e-6, 1e-9, 1e-12])
def test_zero_rows_go_by_their_biases(E, step):
    """Padding rows: every score is 1/2, and the biases lie `step` apart."""
    T, H, K = 12, 256, 8
    x, w, _ = _inputs(T, H, E, 6)
    x[3:] = 0
    bias = (step * torch.randperm(E, generator=torch.Generator().manual_seed(E))).float().cuda()
    bias[5] = bias[9]
    for groups, top_groups in ((1, 1), (8, 3)):
        got = _ids(x, w, K, score="sigmoid", bias=bias, num_groups=groups, top_groups=top_groups)
        assert np.array_equal(got, ids_64(_logits(x, w), "sigmoid", K, bias, groups, top_groups))


@pytest.mark.parametrize("power", [100, -100])
def test_rows_beyond_float32_squares(power):
    """Such rows go by their FP32 logits, here exact: 1 + k 2^-20 times 2^power."""
    T, H, E, K = 9, 256, 256, 8
    k = torch.randperm(E, generator=torch.Generator().manual_seed(1))
    w = torch.zeros(E, H, device="cuda", dtype=torch.bfloat16)
    w[:, 0] = 1
    w[:, 100] = k.cuda().bfloat16()
    x = torch.zeros(T, H, device="cuda", dtype=torch.bfloat16)
    x[:, 0] = 2.0 ** power
    x[:, 100] = 2.0 ** (power - 20)
    for groups, top_groups in ((1, 1), (8, 3)):
        got = _ids(x, w, K, num_groups=groups, top_groups=top_groups)
        assert np.array_equal(got, ids_64(_logits(x, w), "softmax", K, None, groups, top_groups))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_gate_row_leaves_the_others_in_order(bad, score):
    T, H, E, K = 300, 512, 256, 8
    x, _, _ = _inputs(T, H, 1, 9)
    w = _close_gates(H, E, 9)
    w[77, 300] = bad
    for groups, top_groups in ((1, 1), (8, 4)):
        got = _ids(x, w, K, score=score, num_groups=groups, top_groups=top_groups)
        assert np.array_equal(got, ids_64(_logits(x, w), score, K, None, groups, top_groups))


def _cancelling(kind, T, H, E, seed):
    """Rows and gates whose running sums rise far above their logits."""
    x, w, _ = _inputs(T, H, E, seed)
    if kind == "outliers":      # two channels that cancel, at the ends of the row
        x[:, 0], x[:, H - 1] = 4096, -4096
        w[:, 0] = w[:, H - 1] = 1
    elif kind == "neighbours":  # the same inside one K-block
        x[:, 64], x[:, 65 + 16] = 4096, -4096
        w[:, 64] = w[:, 65 + 16] = 1
    else:                       # products of one sign in each half of the row
        half = torch.where(torch.arange(H, device="cuda") < H // 2, 1.0, -1.0).bfloat16()
        x, w = x.abs(), (w.abs() * half)
        w = (w.float() * 0.02 + H ** -0.5 * half.float()).bfloat16()
    return x, w


@pytest.mark.parametrize("kind", ["outliers", "neighbours", "halves"])
@pytest.mark.parametrize("T,H,score", [(9000, 7168, "sigmoid"), (8200, 7168, "softmax"), (5000, 7168, "sigmoid"),
                                       (1100, 7168, "softmax"), (300, 16384, "sigmoid"), (20, 7168, "sigmoid"),
                                       (1, 16384, "softmax")])
def test_sums_that_cancel(T, H, score, kind):
    E, K = 256, 8
    x, w = _cancelling(kind, T, H, E, T)
    got = _ids(x, w, K, score=score)
    assert np.array_equal(got, ids_64(_logits(x, w), score, K))


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("size", [-0.4, -2.0, -20.0, 20.0])
def test_weights_of_far_sigmoid_scores(size, renormalize):
    """Scores down to exp(-2000), together with ordinary ones where ``size`` is
    small: their ratios are ordinary all the same.

    Rows have one element and gates two values, so that the logits are exact.
    A weight is K scores' quotient: exp, sums, quotients and the scale make 32
    half steps, and an exponent of up to 100 that is rounded once (2^-24 of
    it) 100 more.  What is left below 2^-126 has its own steps of 2^-149, times
    the scale."""
    T, H, E, K = 40, 256, 16, 6
    w = torch.zeros(E, H, device="cuda", dtype=torch.bfloat16)
    w[:, 3] = torch.arange(1, E + 1, device="cuda").bfloat16()
    x = torch.zeros(T, H, device="cuda", dtype=torch.bfloat16)
    x[:, 3] = (size * torch.linspace(0.5, 6, T, device="cuda")).bfloat16()
    logits = _logits(x, w)
    r = MoERouter(w, K, max_rows=T, score="sigmoid", renormalize=renormalize, scale=2.5)
    ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
    _, got = r.route(x, ids=ids)
    assert np.array_equal(ids.cpu().numpy(), ids_64(logits, "sigmoid", K))
    l = np.take_along_axis(logits, ids.cpu().numpy().astype(np.int64), axis=1)
    log_score = -np.logaddexp(0.0, -l)
    if renormalize:
        log_score = log_score - np.logaddexp.reduce(log_score, axis=1, keepdims=True)
    want = 2.5 * np.exp(log_score)
    got = got.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= 132 * U * want + 4 * 2.0 ** -149)


@pytest.mark.parametrize("size", [30.0, 3e3, 3e5, 3e8])
def test_large_rows(size):
    """Logits in the hundreds to billions, whose FP32 errors are as large as a
    sigmoid's whole slope."""
    T, H, E, K = 200, 2048, 128, 8
    x, w, b = _inputs(T, H, E, 12, bias=True)
    x = (size * x.float()).bfloat16()
    w[:, 1:] = w[:1, 1:]  # the gates differ in one column
    for groups, top_groups in ((1, 1), (4, 2)):
        got = _ids(x, w, K, score="sigmoid", bias=b, num_groups=groups, top_groups=top_groups)
        assert np.array_equal(got, ids_64(_logits(x, w), "sigmoid", K, b, groups, top_groups))


@pytest.mark.parametrize("E,groups,top_groups", [(257, 1, 1), (384, 3, 2), (384, 12, 5), (510, 5, 2), (512, 16, 3),
                                                 (512, 2, 1), (513, 1, 1), (640, 10, 4), (768, 3, 1), (960, 15, 7),
                                                 (1000, 8, 4), (1024, 1, 1), (1024, 16, 15)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [1, 3, 131])
def test_many_experts_close_together(E, groups, top_groups, score, T):
    """More than 256 experts: a token takes 32 or 64 lanes."""
    H, K = 512, 8
    x, _, b = _inputs(T, H, E, E, bias=score == "sigmoid")
    w = _close_gates(H, E, E)
    bias = None if b is None else 2e-6 * b
    got = _ids(x, w, K, score=score, bias=bias, num_groups=groups, top_groups=top_groups)
    assert np.array_equal(got, ids_64(_logits(x, w), score, K, bias, groups, top_groups))


@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 3)])
@pytest.mark.parametrize("E", [24, 40, 320])
def test_scores_below_float32(E, groups, top_groups):
    """Sigmoids of logits from -100 to -600 are all 0 in float32, not in
    float64."""
    T, H, K = 5, 256, 8
    x = torch.zeros(T, H, device="cuda", dtype=torch.bfloat16)
    x[:, 7] = torch.tensor([-1.0, -2.0, -1.25, -1.5, -1.75], device="cuda").bfloat16()
    w = torch.zeros(E, H, device="cuda", dtype=torch.bfloat16)
    w[:, 7] = (100 + torch.randperm(E, generator=torch.Generator().manual_seed(E)) % 128).cuda().bfloat16()
    x[:, 9], w[:, 9] = 2.0 ** -7, torch.arange(E, device="cuda").bfloat16()  # and experts 2^-7 apart
    got = _ids(x, w, K, score="sigmoid", num_groups=groups, top_groups=top_groups)
    assert np.array_equal(got, ids_64(_logits(x, w), "sigmoid", K, None, groups, top_groups))
