"""64-bit forms of the dense products with bounds on how far a kernel's result
may lie from them, and their inputs.

Bounds count: half a step of bfloat16 (2^-8 of the value) for each rounding to
it; K 2^-24 sum|x w| for FP32 sums of K products in any order; for each FP8
MFMA (rows beyond 16) 2^-10 of its K-block's largest possible product."""

import torch

HALF_BF16 = 2.0 ** -8
FEW = 16  # rows up to which e4m3 products are made on the BF16 MFMA


def blocks(n):
    return -(-n // 128)


def quantise(v, of_rows):
    """e4m3 codes (uint8) and float32 scales of ``v`` per of_rows x 128 block: amax / 448."""
    n, k = v.shape
    nb, kb = -(-n // of_rows), blocks(k)
    p = torch.nn.functional.pad(v.float(), (0, kb * 128 - k, 0, nb * of_rows - n)).view(nb, of_rows, kb, 128)
    amax = p.abs().amax(dim=(1, 3), keepdim=True)
    s = amax / torch.full_like(amax, 448.0)
    q = torch.where(s > 0, p / torch.where(s > 0, s, 1.0), 0.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(nb * of_rows, kb * 128)[:n, :k].contiguous(), s.view(nb, kb).contiguous()


def values(codes, scale, of_rows):
    n, k = codes.shape
    f = scale.double().repeat_interleave(of_rows, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return codes.view(torch.float8_e4m3fn).double() * f


def product64(x, xs, w, ws):
    """x w^T from codes and scales, and the bound of its FP32 form."""
    a, b = values(x, xs, 1), values(w, ws, 128)
    y = a @ b.T
    err = x.shape[1] * 2.0 ** -24 * (a.abs() @ b.abs().T)
    if len(x) > FEW:
        def tops(v):  # largest of each row's K-blocks
            k = v.shape[1]
            return torch.nn.functional.pad(v.abs(), (0, blocks(k) * 128 - k)).view(len(v), -1, 128).amax(2)
        err = err + 2.0 ** -10 * (tops(a) @ tops(b).T)
    return y, err


def rounded(y, err, add=None):
    """Bound after the addition of ``add`` and one rounding to bfloat16."""
    if add is not None:
        y = y + add.double()
        err = err + 2.0 ** -24 * y.abs()
    return y, err + HALF_BF16 * (y.abs() + err) + 2.0 ** -133


def swiglu64(g, u, eg, eu):
    """h and its bound from bounds on g and u: |silu'| <= 1.1, and 2^-18 for the
    hardware's exponential and reciprocal."""
    s = torch.sigmoid(g)
    h = g * s * u
    return h, 1.1 * u.abs() * eg + (g * s).abs() * eu + 1.1 * eg * eu + 2.0 ** -18 * h.abs()


def e4m3(v):
    """Nearest e4m3 value of float64 v, ties to even."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return (torch.round(v / step) * step).clamp(-448, 448)


def shared64(x, xs, w13, s13, w2, s2, add=None):
    """The shared expert.  A code of h may be any between those of its quotient
    less and plus its error."""
    T, I = len(x), w2.shape[1]
    gu, e = product64(x, xs, w13, s13)
    h, eh = swiglu64(gu[:, :I], gu[:, I:], e[:, :I], e[:, I:])
    b, eb = h.view(T, -1, 128), eh.view(T, -1, 128)
    top = b.abs().amax(2, keepdim=True)
    s = top / 448
    es = (eb.amax(2, keepdim=True) / top.clamp(min=1e-300)).clamp(max=1.0) + 2.0 ** -22  # relative
    q = b / s.clamp(min=1e-300)
    eq = eb / s.clamp(min=1e-300) + q.abs() * es
    code, low, high = e4m3(q), e4m3(q - eq), e4m3(q + eq)
    v = code * s
    ev = torch.maximum(high - code, code - low) * s + torch.maximum(high.abs(), low.abs()) * s * es
    w = values(w2, s2, 128)
    v, ev = v.reshape(T, I), ev.reshape(T, I)
    y = v @ w.T
    err = ev @ w.abs().T + product64_error(v, w, T)
    return rounded(y, err, add)


def product64_error(a, b, rows):
    err = a.shape[1] * 2.0 ** -24 * (a.abs() @ b.abs().T)
    if rows > FEW:
        ta, tb = (v.abs().view(len(v), -1, 128).amax(2) for v in (a, b))
        err = err + 2.0 ** -10 * (ta @ tb.T)
    return err


def ffn64(x, w13, w2, dy=None):
    """The BF16 block: {name: (value, bound)} of y, and of the gradients."""
    x, w13, w2 = x.detach().double(), w13.detach().double(), w2.detach().double()
    I, u24 = w2.shape[1], 2.0 ** -24
    gu, eg = x @ w13.T, w13.shape[1] * u24 * (x.abs() @ w13.abs().T)
    g, u = gu[:, :I], gu[:, I:]
    h, eh = swiglu64(g, u, eg[:, :I], eg[:, I:])
    eh = eh + HALF_BF16 * (h.abs() + eh)
    out = {"y": rounded(h @ w2.T, eh @ w2.abs().T + I * u24 * (h.abs() @ w2.abs().T))}
    if dy is None:
        return out
    dy = dy.double()
    dh, edh = dy @ w2, len(w2) * u24 * (dy.abs() @ w2.abs())
    s = torch.sigmoid(g)
    silu, slope = g * s, s * (1 + g * (1 - s))
    du, dg = dh * silu, dh * u * slope
    # |silu''| <= 1/2, |silu'| <= 1.1; the hardware's functions
    rg, ru = eg[:, :I], eg[:, I:]
    edu = 1.1 * edh * g.abs() + dh.abs() * 1.1 * rg + 2.0 ** -18 * (dh * g).abs()
    edg = 1.1 * edh * u.abs() + dh.abs() * (0.5 * u.abs() * rg + 1.1 * ru) + 2.0 ** -16 * (dh * u).abs()
    edu, edg = edu + HALF_BF16 * (du.abs() + edu), edg + HALF_BF16 * (dg.abs() + edg)
    d, ed = torch.cat((dg, du), 1), torch.cat((edg, edu), 1)

    def product(a, ea, b):
        k = a.shape[1]
        return a @ b, ea @ b.abs() + k * u24 * (a.abs() @ b.abs())

    out["dx"] = rounded(*product(d, ed, w13))
    out["dw13"] = product(d.T, ed.T, x)
    dw2 = dy.T @ h
    out["dw2"] = dw2, dy.abs().T @ eh + len(dy) * u24 * (dy.abs().T @ h.abs())
    return out


def assert_within(got, want, bound, what):
    got = got.double()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond their bounds, first at "
                           f"{tuple(bad.nonzero()[0].tolist())}: {got[bad][0].item()} for {want[bad][0].item()} +- "
                           f"{bound[bad][0].item()}")


def rel_rms(got, want):
    return float((got.double() - want).square().mean().sqrt() / want.square().mean().sqrt().clamp(min=1e-300))


def fp8_inputs(m, n, k, seed, device="cuda"):
    gen = torch.Generator(device=device).manual_seed(seed)
    x, xs = quantise(torch.randn(m, k, generator=gen, device=device), 1)
    w, ws = quantise(torch.randn(n, k, generator=gen, device=device) * k ** -0.5, 128)
    return x, xs, w, ws


def ffn_inputs(t, h, i, seed, device="cuda"):
    gen = torch.Generator(device=device).manual_seed(seed)

    def rnd(*shape, f=1.0):
        return (torch.randn(*shape, generator=gen, device=device) * f).bfloat16()

    return rnd(t, h), rnd(2 * i, h, f=h ** -0.5), rnd(h, i, f=i ** -0.5), rnd(t, h)
