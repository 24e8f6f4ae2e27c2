"""The few-token layer held to a bound on every element, made from its
arithmetic and the float64 values of the case.

u = 2^-24.  FC1 and FC2 multiply exact e4m3 (or MX, BF16) products on the BF16
MFMA: one instruction errs by at most 3u of its partial sum and 8u of its
largest product, a K-block is four of them, and scaling and adding the blocks
and the waves' parts is a rounding each.  With s = sum |products| (scaled) over
all of K that is
    gamma s,  gamma = (4 (3 + 8) + 3 + K / 128 + 8 + 2) u.
h = silu(g) u moves by |silu'| <= 1.1 times g's error, silu(g) times u's, and 8u
of its own (exp, quotient, products).  A code of h may be any within its
quotient's error (h's, and the scale's: that of the block's largest |h|, 4u
with the divisions); a BF16 h likewise.  These make FC2's input error, which
comes out weighted with |W2|, FC2's own gamma, (K + 16) u for the experts'
sum, and at last half a step of BF16.
"""

import numpy as np
import pytest
import torch

from oracle import formats, moe_ref
from tests.test_gpu_decode import _bits, _setup, _setup_mx

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_ffn_route_amd.harness import make_layer, to_device

U = 2.0 ** -24


def _gamma(k):
    return (4 * (3 + 8) + 3 + k / 128 + 8 + 2) * U


def _expected(x, inp, mx, left=None):
    """(output in float64, bound on the error of each element).  left: the
    columns of h whose errors W2 does not cancel, where its other products do
    (in every aligned eight columns: no partial sum is above 17 of them)."""
    T, H = x.shape
    I, K = inp.w2.shape[2], inp.topk_idx.shape[1]
    out, err = np.zeros((T, H)), np.zeros((T, H))
    for e in range(inp.w13.shape[0]):
        t, k = np.nonzero(inp.topk_idx == e)
        if t.size == 0:
            continue
        if mx:
            w13, w2 = (moe_ref.dequant_mx(a[e], s[e], mx) for a, s in ((inp.w13, inp.w13_scale), (inp.w2, inp.w2_scale)))
        else:
            w13, w2 = (moe_ref.dequant_block128(a[e], s[e])
                       for a, s in ((inp.w13, inp.w13_scale), (inp.w2, inp.w2_scale)))
        gu, dgu = x[t] @ w13.T, _gamma(H) * (np.abs(x[t]) @ np.abs(w13).T)
        g, u = gu[:, :I], gu[:, I:]
        h = moe_ref.silu(g) * u
        dh = 1.1 * np.abs(u) * dgu[:, :I] + np.abs(moe_ref.silu(g)) * dgu[:, I:] + 8 * U * np.abs(h)
        if mx:
            hq = formats.bf16_bits_to_f64(formats.bf16_rne_bits(h))
            lo, hi = (formats.bf16_bits_to_f64(formats.bf16_rne_bits(h + d)) for d in (-dh, dh))
            dhq = np.maximum(hi - hq, hq - lo)
        else:
            b, db = h.reshape(-1, I // 128, 128), dh.reshape(-1, I // 128, 128)
            top = np.abs(b).max(axis=2, keepdims=True)
            scale = top / 448.0
            ds = db.max(axis=2, keepdims=True) / top + 4 * U
            q, dq = b / scale, (db / scale + np.abs(b / scale) * ds)
            code, lo, hi = (formats.e4m3_decode(formats.e4m3_encode_rne_sat(v)) for v in (q, q - dq, q + dq))
            hq = (code * scale).reshape(h.shape)
            dhq = ((np.maximum(hi - code, code - lo) + np.maximum(np.abs(lo), np.abs(hi)) * ds) * scale).reshape(h.shape)
        y, sy = hq @ w2.T, np.abs(hq) @ np.abs(w2).T
        if left is None:
            dy = dhq @ np.abs(w2).T + _gamma(I) * sy
        else:
            top = np.abs(hq).reshape(-1, I // 128, 128).max(axis=2).sum(axis=1)[:, None] * np.abs(w2).max()
            dy, sy = dhq[:, left] @ np.abs(w2[:, left]).T + 4 * (3 * 17 + 8) * U * top, \
                np.abs(hq[:, left]) @ np.abs(w2[:, left]).T
            dy += _gamma(I) * sy
        rw = inp.topk_w[t, k][:, None].astype(np.float64)
        np.add.at(out, t, rw * y)
        np.add.at(err, t, np.abs(rw) * (dy + (K + 16) * U * sy))
    return out, err + 2.0 ** -8 * (np.abs(out) + err)


@pytest.mark.parametrize("T,H,I,E,K", [(1, 512, 256, 8, 2), (5, 2048, 768, 16, 6), (16, 1024, 384, 16, 8),
                                       (8, 256, 2048, 4, 2), (3, 7168, 256, 8, 4), (5, 10496, 256, 4, 2),
                                       (8, 16384, 128, 4, 2)])
@pytest.mark.parametrize("form", ["codes", "e4m3", "e5m2"])
def test_every_element(T, H, I, E, K, form):
    if form == "codes":
        inp, dev, layer = _setup(T, H, I, E, K, seed=T + 40)
        layer.stage(dev.x, dev.topk_idx, dev.topk_w)
        codes = layer.region("xq", torch.uint8, (T, H)).clone()
        scale = layer.region("xs", torch.float32, (T, H // 128)).clone()
        got = layer.decode(codes, dev.topk_idx, dev.topk_w, x_scale=scale)
        x = moe_ref.dequant_rows_1x128(codes.cpu().numpy(), scale.cpu().numpy())
    else:
        inp, dev, layer = _setup_mx(T, H, I, E, K, form, seed=T + 40)
        got = layer.decode(dev.x, dev.topk_idx, dev.topk_w)
        x = formats.bf16_bits_to_f64(inp.x_bf16)
    want, bound = _expected(x, inp, None if form == "codes" else form)
    err = np.abs(formats.bf16_bits_to_f64(_bits(got)) - want)
    print("largest error / bound %.3f, median bound / |out| %.4f" % ((err / bound).max(),
                                                                     np.median(bound / np.maximum(np.abs(want), 1e-30))))
    assert np.all(err <= bound)


def test_fc2_terms_beside_large_ones_that_cancel():
    """All columns of h are equal; of every eight, W2 takes four with +448 and
    four with -448, but for one pair of a K-block: what is left is one product
    2^-12.8 of the others."""
    T, H, I, E, K = 4, 512, 512, 4, 2
    inp, _, _ = _setup(T, H, I, E, K, seed=77)
    inp.w13[:, :I], inp.w13[:, I:] = inp.w13[:, :1], inp.w13[:, I:I + 1]
    inp.w13_scale[:, :I // 128], inp.w13_scale[:, I // 128:] = inp.w13_scale[:, :1], inp.w13_scale[:, I // 128:I // 128 + 1]
    rng = np.random.default_rng(5)
    value = np.concatenate([rng.permutation([448.0] * 4 + [-448.0] * 4) for _ in range(I // 8)])
    left = np.zeros(I, dtype=bool)
    for b in range(0, I, 128):
        at = b + 8 * rng.integers(16)
        plus, minus = at + np.argmax(value[at:at + 8]), at + np.argmin(value[at:at + 8])
        value[plus], value[minus] = 2.0 ** -4, 0.0
        left[[plus, minus]] = True
    inp.w2[:] = formats.e4m3_encode_rne_sat(value)[None, None, :]
    dev = to_device(inp)
    layer = make_layer(inp.shape, dev)
    layer.stage(dev.x, dev.topk_idx, dev.topk_w)
    codes = layer.region("xq", torch.uint8, (T, H)).clone()
    scale = layer.region("xs", torch.float32, (T, H // 128)).clone()
    got = layer.decode(codes, dev.topk_idx, dev.topk_w, x_scale=scale)
    want, bound = _expected(moe_ref.dequant_rows_1x128(codes.cpu().numpy(), scale.cpu().numpy()), inp, None, left)
    err = np.abs(formats.bf16_bits_to_f64(_bits(got)) - want)
    print("largest error / bound %.3f, median bound / |out| %.4f" % ((err / bound).max(), np.median(bound / np.abs(want))))
    assert np.all(err <= bound)
