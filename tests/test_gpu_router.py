"""The router (moe_router_*) against its formula in float64.

Expert ids are compared for equality: the router promises those of 64-bit
arithmetic.  A weight is compared within the logits' error: the margin below
which the router recomputes, 2^-17 (|x| max|w| / sqrt(H) + max|l|), bounds a
logit's error dl; a sigmoid or softmax score changes by at most dl (softmax:
2 dl) of itself, a renormalised weight by twice that, and exp, division, sum
and scale add a few steps of 2^-24 (32 taken).
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_ffn_route_amd import MoEError, MoERouter

U = 2.0 ** -24


def reference(x, w, top_k, score, bias=None, groups=1, top_groups=1, renormalize=True, scale=1.0):
    """(ids [T, K], weights [T, K], relative bound on the weights [T, 1]) in float64."""
    x, w = x.double().cpu().numpy(), w.double().cpu().numpy()
    T, E = x.shape[0], w.shape[0]
    logits = x @ w.T
    if score == "softmax":
        z = np.exp(logits - logits.max(axis=1, keepdims=True))
        s, choice = z / z.sum(axis=1, keepdims=True), logits.copy()
    else:
        s = 1.0 / (1.0 + np.exp(-logits))
        choice = s + (0.0 if bias is None else bias.double().cpu().numpy())
    if top_groups < groups:
        n = E // groups
        by = np.sort(choice.reshape(T, groups, n), axis=2)[:, :, ::-1]
        value = by[:, :, 0] if score == "softmax" or n == 1 else by[:, :, 0] + by[:, :, 1]
        order = np.argsort(-value, axis=1, kind="stable")[:, :top_groups]
        keep = np.zeros((T, groups), dtype=bool)
        np.put_along_axis(keep, order, True, axis=1)
        choice = np.where(np.repeat(keep, n, axis=1), choice, -np.inf)
    ids = np.argsort(-choice, axis=1, kind="stable")[:, :top_k]
    wt = np.take_along_axis(s, ids, axis=1)
    if renormalize:
        wt = wt / wt.sum(axis=1, keepdims=True)
    dl = 2.0 ** -17 * (np.linalg.norm(x, axis=1) * np.linalg.norm(w, axis=1).max() / np.sqrt(x.shape[1])
                       + np.abs(logits).max(axis=1))
    return ids, wt * scale, (4 * dl + 32 * U)[:, None]


def check(router, x, ref, base=0, local=None, **kw):
    T = x.shape[0]
    ids, wt, tol = ref
    local = kw["experts"] - base if local is None else local
    got_ids = torch.full(ids.shape, -7, dtype=torch.int32, device="cuda")
    idx, w = router.route(x, ids=got_ids)
    assert np.array_equal(got_ids.cpu().numpy(), ids)
    here = (ids >= base) & (ids < base + local)
    assert np.array_equal(idx.cpu().numpy(), np.where(here, ids - base, -1))
    w = w.double().cpu().numpy()
    assert np.all(np.abs(w - wt) <= tol * np.abs(wt) + 2.0 ** -140)


def _inputs(T, H, E, seed, bias=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w = (torch.randn(E, H, generator=g, device="cuda") * H ** -0.5).bfloat16()
    b = 0.1 * torch.randn(E, generator=g, device="cuda") if bias else None
    return x, w, b


@pytest.mark.parametrize("E,K,groups,top_groups", [
    (1, 1, 1, 1), (2, 2, 1, 1), (8, 8, 1, 1), (31, 6, 1, 1), (32, 6, 1, 1), (33, 8, 3, 2), (64, 4, 16, 5),
    (65, 8, 5, 2), (100, 8, 4, 3), (128, 8, 8, 4), (200, 7, 8, 1), (256, 8, 8, 4), (256, 8, 1, 1), (257, 8, 1, 1),
    (512, 8, 16, 3), (640, 8, 10, 4), (1000, 8, 8, 4), (1024, 8, 16, 15), (1023, 8, 1, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,H", [(1, 128), (70, 384)])
def test_experts_groups_and_scores(T, H, E, K, groups, top_groups, score):
    x, w, b = _inputs(T, H, E, E * 3 + T, bias=score == "sigmoid")
    base, local = E // 3, max(1, E // 2)
    r = MoERouter(w, K, max_rows=T, score=score, bias=b, num_groups=groups, top_groups=top_groups, scale=2.5,
                  expert_base=base, local_experts=local)
    check(r, x, reference(x, w, K, score, b, groups, top_groups, scale=2.5), base, local, experts=E)


@pytest.mark.parametrize("T", [1, 15, 16, 17, 32, 33, 1023, 1024, 1025, 8192, 8193])
@pytest.mark.parametrize("H,E", [(128, 40), (1024, 64), (2048, 256)])
def test_batch_sizes(T, H, E):
    x, w, b = _inputs(T, H, E, T + H, bias=True)
    r = MoERouter(w, 8, max_rows=T, score="sigmoid", bias=b, num_groups=4, top_groups=2)
    check(r, x, reference(x, w, 8, "sigmoid", b, 4, 2), experts=E)


@pytest.mark.parametrize("T", [512, 513, 4097, 8192, 8193, 9001])
@pytest.mark.parametrize("E,K", [(8, 2), (32, 6), (60, 8), (300, 8)])
def test_expert_tiles_and_batches(T, E, K):
    """One block of experts, two, and more than one workgroup holds."""
    x, w, _ = _inputs(T, 512, E, T + E)
    r = MoERouter(w, K, max_rows=T)
    check(r, x, reference(x, w, K, "softmax"), experts=E)


@pytest.mark.parametrize("T,H", [(3, 7168), (300, 7168), (2500, 7168), (5, 16384), (1100, 16384)])
def test_long_rows(T, H):
    x, w, b = _inputs(T, H, 256, T + H, bias=True)
    r = MoERouter(w, 8, max_rows=T, score="sigmoid", bias=b, num_groups=8, top_groups=4)
    check(r, x, reference(x, w, 8, "sigmoid", b, 8, 4), experts=256)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_without_renormalisation(score):
    x, w, _ = _inputs(90, 512, 48, 2)
    r = MoERouter(w, 4, max_rows=128, score=score, renormalize=False)
    check(r, x, reference(x, w, 4, score, renormalize=False), experts=48)


def test_logit_error_has_room_below_the_margin():
    """log(w_i / w_j) of unnormalised softmax weights is l_i - l_j: the FP32
    product's error, at the longest sums one accumulator takes (one K part),
    has to stay far below the margin that makes the ids exact."""
    T, H, E = 33000, 16384, 256
    x, w, _ = _inputs(2000, H, E, 5)
    xs = x.repeat(17, 1)[:T].contiguous()
    r = MoERouter(w, 8, max_rows=T)
    idx, wt = r.route(xs)
    for at in (slice(0, 2000), slice(32000, 33000)):
        rows = xs[at].double().cpu().numpy()
        logits = rows @ w.double().cpu().numpy().T
        l = np.take_along_axis(logits, idx[at].cpu().numpy(), axis=1)
        lw = np.log(wt[at].double().cpu().numpy())
        err = np.abs((lw - lw[:, :1]) - (l - l[:, :1]))
        margin = 2.0 ** -17 * (np.linalg.norm(rows, axis=1) / np.sqrt(H) + np.abs(logits).max(axis=1))
        print("largest logit error: %.3g, smallest margin %.3g" % (err.max(), margin.min()))
        # 2 dl for a difference; expf and division cost a few 2^-24
        assert np.all(err <= 2 * margin[:, None] / 8 + 8 * U)


@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("H", [256, 7168])
def test_near_ties_are_decided_in_64_bits(H, score, groups, top_groups):
    """Experts that differ in a few small elements only: their logits are
    closer than FP32 can tell."""
    T, E, K = 65, 64, 8
    x, w, _ = _inputs(T, H, 1, H)
    w = w.expand(E, H).clone()
    g = torch.Generator(device="cuda").manual_seed(1)
    at = torch.randint(0, H, (E, 4), generator=g, device="cuda")
    tiny = (1e-7 * torch.randn(E, 4, generator=g, device="cuda")).bfloat16()
    w.scatter_(1, at, tiny)
    w[:, :8] = tiny[:, :1]  # every expert's own tiny elements in the same columns
    r = MoERouter(w, K, max_rows=T, score=score, num_groups=groups, top_groups=top_groups)
    check(r, x, reference(x, w, K, score, None, groups, top_groups), experts=E)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_exact_ties_go_to_the_lowest_expert(score):
    x, w, _ = _inputs(40, 512, 48, 3)
    w[1::3] = w[0::3]
    w[2::3] = w[0::3]      # every expert three times
    x[7] = 0               # every logit 0
    for groups, top_groups in ((1, 1), (4, 2)):
        r = MoERouter(w, 8, max_rows=40, score=score, num_groups=groups, top_groups=top_groups)
        ids = torch.empty(40, 8, dtype=torch.int32, device="cuda")
        r.route(x, ids=ids)
        assert ids[7].tolist() == list(range(8))
        check(r, x[:7], tuple(v[:7] for v in reference(x, w, 8, score, None, groups, top_groups)), experts=48)
        check(r, x[8:], tuple(v[8:] for v in reference(x, w, 8, score, None, groups, top_groups)), experts=48)


def test_large_common_part():
    """Logits of one sign and size (about 60 of |x| |w| = 100): their FP32
    steps are far above the differences' own."""
    T, H, E = 500, 4096, 64
    x, w, _ = _inputs(T, H, E, 8)
    x = x.abs()
    w = (w.float() * 0.1 + 0.02).bfloat16()
    r = MoERouter(w, 8, max_rows=T)
    check(r, x, reference(x, w, 8, "softmax"), experts=E)


def test_same_experts_alone_and_in_a_batch():
    T, H, E = 1500, 2048, 128
    x, w, b = _inputs(T, H, E, 11, bias=True)
    r = MoERouter(w, 8, max_rows=T, score="sigmoid", bias=b, num_groups=8, top_groups=4)
    whole, _ = r.route(x)
    for t in (0, 1, 700, 1499):
        assert torch.equal(r.route(x[t:t + 1])[0], whole[t:t + 1])
    assert torch.equal(r.route(x[100:140])[0], whole[100:140])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_rows_touch_no_other(bad):
    T, H, E = 20, 256, 40
    x, w, _ = _inputs(T, H, E, 4)
    for score, groups, tg in (("softmax", 1, 1), ("sigmoid", 4, 2)):
        r = MoERouter(w, 6, max_rows=T, score=score, num_groups=groups, top_groups=tg)
        clean_idx, clean_w = r.route(x)
        y = x.clone()
        y[9, 17] = bad
        idx, wt = r.route(y)
        keep = torch.arange(T, device="cuda") != 9
        assert torch.equal(idx[keep], clean_idx[keep]) and torch.equal(wt[keep], clean_w[keep])
        got = idx[9].tolist()
        assert len(set(got)) == 6 and min(got) >= 0 and max(got) < E
    # every logit NaN: the lowest experts, weights that the layer's checks mask
    y[9] = float("nan")
    r = MoERouter(w, 6, max_rows=T)
    idx, wt = r.route(y)
    assert idx[9].tolist() == [0, 1, 2, 3, 4, 5] and torch.isnan(wt[9]).all()


def test_rows_with_a_stride_and_buffers_left_alone():
    T, H, E = 37, 512, 64
    x, w, _ = _inputs(T, H, E, 6)
    wide = torch.full((T, H + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :H] = x
    r = MoERouter(w, 4, max_rows=50)
    idx, wt = r.route(x)
    big_i = torch.full((T + 3, 4), -9, dtype=torch.int32, device="cuda")
    big_w = torch.full((T + 3, 4), -9.0, device="cuda")
    r.route(wide[:, :H], big_i[:T], big_w[:T])
    assert torch.equal(big_i[:T], idx) and torch.equal(big_w[:T], wt)
    assert (big_i[T:] == -9).all() and (big_w[T:] == -9).all()
    empty = r.route(x[:0])
    assert empty[0].shape == (0, 4)


def test_stream_and_graph_replays():
    T, H, E = 50, 1024, 256
    x, w, b = _inputs(T, H, E, 7, bias=True)
    r = MoERouter(w, 8, max_rows=T, score="sigmoid", bias=b, num_groups=8, top_groups=4)
    e = MoERouter(w, 8, max_rows=T, score="sigmoid", bias=b, num_groups=8, top_groups=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    idx = torch.empty(T, 8, dtype=torch.int32, device="cuda")
    wt = torch.empty(T, 8, device="cuda")
    with torch.cuda.stream(side):
        r.route(x, idx, wt)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            r.route(x, idx, wt)
    torch.cuda.synchronize()
    for seed in (1, 2, 3):
        x.copy_(_inputs(T, H, E, seed)[0])
        want = e.route(x)
        idx.fill_(-5)
        wt.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, want[0]) and torch.equal(wt, want[1])


def test_refusals():
    x, w, b = _inputs(8, 256, 16, 1, bias=True)
    r = MoERouter(w, 4, max_rows=8)
    for bad in (x.float(), x[:, :128], x.cpu(), x.t().contiguous().t()):
        with pytest.raises(ValueError):
            r.route(bad)
    with pytest.raises(ValueError):
        r.route(x, torch.empty(8, 4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        r.route(x, ids=torch.empty(8, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(MoEError):
        r.route(torch.zeros(9, 256, dtype=torch.bfloat16, device="cuda"))  # above max_rows
    with pytest.raises(MoEError):
        r.route(x[:1].expand(8, 256))
    with pytest.raises(MoEError):
        MoERouter(w, 4, max_rows=8, bias=b)            # softmax with a bias
    with pytest.raises(ValueError):
        MoERouter(w.float(), 4, max_rows=8)
    with pytest.raises(ValueError):
        MoERouter(w, 4, max_rows=8, score="relu")
    with pytest.raises(ValueError):
        MoERouter(w, 4, max_rows=8, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
