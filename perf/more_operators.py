"""Cases of the dense operators beside the routed experts: the e4m3 matrix
product with block scales, the shared expert (a gated feed-forward block on
that product) and the BF16 gated feed-forward block with its gradients.

``run`` computes them in elementary torch operations where ``own`` is false
and through this package where it is true; ``exact`` computes them from their
definition in 64 bits.
"""

import torch

own = False

E4M3_MAX = 448.0
LARGEST = {"linear": 16384 * 7168 * 7168, "shared": 32768 * 7168 * 2048, "ffn": 16384 * 7168 * 2048,
           "train": 4096 * 7168 * 2048}


def listed():
    return [
        # one token being decoded, the down projection of a DeepSeek-V3-like shared expert: its weights are all there is
        {"name": "linear_one", "op": "linear", "tokens": 1, "rows": 7168, "cols": 2048, "add": False},
        # a ragged batch through a projection whose last weight blocks are cut in both directions, onto a residual
        {"name": "linear_ragged", "op": "linear", "tokens": 301, "rows": 1003, "cols": 2000, "add": True},
        # sequences decoded together through a square projection
        {"name": "linear_batch", "op": "linear", "tokens": 64, "rows": 7168, "cols": 7168, "add": False},
        # a large prompt through the same projection
        {"name": "linear_large", "op": "linear", "tokens": 16384, "rows": 7168, "cols": 7168, "add": False},
        # the shared expert of one token being decoded, added to the routed experts' output
        {"name": "shared_one", "op": "shared", "tokens": 1, "hidden": 7168, "intermediate": 2048, "add": True},
        # a mid-size decode batch of a small model
        {"name": "shared_small", "op": "shared", "tokens": 77, "hidden": 2048, "intermediate": 768, "add": True},
        # a prompt through the shared expert
        {"name": "shared_prompt", "op": "shared", "tokens": 4096, "hidden": 7168, "intermediate": 2048, "add": True},
        # the largest batch of the layer's own token sweep
        {"name": "shared_large", "op": "shared", "tokens": 32768, "hidden": 7168, "intermediate": 2048, "add": False},
        # the BF16 block for one token (a model before its quantisation)
        {"name": "ffn_one", "op": "ffn", "tokens": 1, "hidden": 7168, "intermediate": 2048, "train": False},
        # a forward pass of a large batch, as an evaluation makes it
        {"name": "ffn_large", "op": "ffn", "tokens": 16384, "hidden": 7168, "intermediate": 2048, "train": False},
        # a training step's pass over a short ragged batch of a small model, odd sizes
        {"name": "train_ragged", "op": "ffn", "tokens": 301, "hidden": 2040, "intermediate": 776, "train": True},
        # a training step's pass over one sequence of 4096 tokens
        {"name": "train_sequence", "op": "ffn", "tokens": 4096, "hidden": 7168, "intermediate": 2048, "train": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("linear", "shared", "ffn", "train"))
    if op == "linear":
        rows, cols = _log_int(rng, 64, 16384), 16 * _log_int(rng, 8, 1024)
        tokens = _log_int(rng, 1, min(16384, LARGEST[op] // (rows * cols)))
        return {"op": op, "tokens": tokens, "rows": rows, "cols": cols, "add": rng.random() < 0.5}
    step = 128 if op == "shared" else 8
    hidden = step * rng.randint(256 // step, 8192 // step)
    intermediate = step * _log_int(rng, 128 // step, 8192 // step)
    tokens = _log_int(rng, 1, min(32768 if op == "shared" else 16384, LARGEST[op] // (hidden * intermediate)))
    case = {"op": "shared" if op == "shared" else "ffn", "tokens": tokens, "hidden": hidden,
            "intermediate": intermediate}
    case["add" if op == "shared" else "train"] = rng.random() < 0.5 if op == "shared" else op == "train"
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


def _blocks(n):
    return -(-n // 128)


def _pad(v, rows, cols):
    return torch.nn.functional.pad(v, (0, cols - v.shape[1], 0, rows - v.shape[0]))


def _codes(v, dims):
    """e4m3 values and scales of ``v`` over the blocks that ``dims`` spans: amax / 448."""
    amax = v.abs().amax(dim=dims, keepdim=True)
    scale = amax / torch.full_like(amax, E4M3_MAX)  # by a Python number, torch multiplies with a rounded 1 / 448
    q = torch.where(scale > 0, v / torch.where(scale > 0, scale, 1.0), 0.0).clamp(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn), scale


def _fp8_weight(n, k, gen):
    """Codes [n, k] of N(0, 1/k) and a scale per 128 x 128 block."""
    nb, kb = _blocks(n), _blocks(k)
    w = torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5
    q, s = _codes(_pad(w, nb * 128, kb * 128).view(nb, 128, kb, 128), (1, 3))
    return q.view(torch.uint8).view(nb * 128, kb * 128)[:n, :k].contiguous(), s.view(nb, kb).contiguous()


def _fp8_rows(t, k, gen):
    """Activation rows as codes [t, k] and a scale per 128 columns; a few columns are much larger than the rest."""
    kb = _blocks(k)
    x = torch.randn(t, k, generator=gen, device="cuda")
    x *= 1.0 + 7.0 * (torch.rand(k, generator=gen, device="cuda") < 0.01)
    q, s = _codes(_pad(x, t, kb * 128).view(t, kb, 128), (2,))
    return q.view(torch.uint8).view(t, kb * 128)[:, :k].contiguous(), s.view(t, kb).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    T = case["tokens"]
    if case["op"] == "linear":
        s["x"], s["x_scale"] = _fp8_rows(T, case["cols"], gen)
        s["w"], s["w_scale"] = _fp8_weight(case["rows"], case["cols"], gen)
        s["onto"] = torch.randn(T, case["rows"], generator=gen, device="cuda").bfloat16() if case["add"] else None
        return s
    H, I = case["hidden"], case["intermediate"]
    if case["op"] == "shared":
        s["x"], s["x_scale"] = _fp8_rows(T, H, gen)
        s["w13"], s["w13_scale"] = _fp8_weight(2 * I, H, gen)
        s["w2"], s["w2_scale"] = _fp8_weight(H, I, gen)
        s["onto"] = torch.randn(T, H, generator=gen, device="cuda").bfloat16() if case["add"] else None
        if own:
            from mixture_experts_ffn_route_amd import MoESharedExpert
            s["shared"] = MoESharedExpert(s["w13"], s["w13_scale"], s["w2"], s["w2_scale"])
        return s
    s["x"] = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
    s["w13"] = (torch.randn(2 * I, H, generator=gen, device="cuda") * H ** -0.5).bfloat16()
    s["w2"] = (torch.randn(H, I, generator=gen, device="cuda") * I ** -0.5).bfloat16()
    if case["train"]:
        s["dy"] = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
        for name in ("x", "w13", "w2"):
            s[name].requires_grad_(True)
    return s


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------


def _weight(codes, scale):
    n, k = codes.shape
    f = scale.repeat_interleave(128, dim=0)[:n].repeat_interleave(128, dim=1)[:, :k]
    return codes.view(torch.float8_e4m3fn).float() * f


def _rows(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(128, dim=1)[:, :codes.shape[1]]


def _onto(y, onto):
    return (y if onto is None else y + onto.float()).bfloat16()


def _linear(s):
    return _onto(_rows(s["x"], s["x_scale"]) @ _weight(s["w"], s["w_scale"]).t(), s["onto"])


def _shared(s):
    T, I = s["tokens"], s["intermediate"]
    gu = _rows(s["x"], s["x_scale"]) @ _weight(s["w13"], s["w13_scale"]).t()
    h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
    q, f = _codes(h.view(T, I // 128, 128), (2,))
    return _onto((q.float() * f).view(T, I) @ _weight(s["w2"], s["w2_scale"]).t(), s["onto"])


def _ffn(s):
    I = s["intermediate"]
    x, w13, w2 = (s[name].detach().float() for name in ("x", "w13", "w2"))
    gu = x @ w13.t()
    g, u = gu[:, :I], gu[:, I:]
    sig = torch.sigmoid(g)
    silu = g * sig
    h = silu * u
    out = {"y": (h @ w2.t()).bfloat16()}
    if s["train"]:
        dy = s["dy"].float()
        dh = dy @ w2
        dgu = torch.cat((dh * u * sig * (1.0 + g * (1.0 - sig)), dh * silu), dim=1)
        out["dx"] = (dgu @ w13).bfloat16()
        out["dw13"] = (dgu.t() @ x).bfloat16()
        out["dw2"] = (dy.t() @ h).bfloat16()
    return out


def run(s):
    if s["op"] == "linear":
        if not own:
            return _linear(s)
        from mixture_experts_ffn_route_amd import fp8_matmul
        return fp8_matmul(s["x"], s["x_scale"], s["w"], s["w_scale"], add=s["onto"])
    if s["op"] == "shared":
        if not own:
            return _shared(s)
        return s["shared"].forward(s["x"], s["x_scale"], add=s["onto"])
    if not own:
        return _ffn(s)
    from mixture_experts_ffn_route_amd import gated_ffn
    y = gated_ffn(s["x"], s["w13"], s["w2"])
    if not s["train"]:
        return {"y": y}
    dx, dw13, dw2 = torch.autograd.grad(y, (s["x"], s["w13"], s["w2"]), s["dy"])
    return {"y": y.detach(), "dx": dx, "dw13": dw13, "dw2": dw2}


def work(case):
    T = case["tokens"]
    if case["op"] == "linear":
        n, k = case["rows"], case["cols"]
        scales = 4 * _blocks(k) * (T + _blocks(n))
        return {"bytes": (T + n) * k + scales + (4 if case["add"] else 2) * T * n, "flops": 2 * T * n * k}
    H, I = case["hidden"], case["intermediate"]
    if case["op"] == "shared":
        weights = 3 * H * I * (1 + 4 / 16384)
        return {"bytes": T * H * (1 + 4 / 128) + weights + (4 if case["add"] else 2) * T * H, "flops": 6 * T * H * I}
    if case["train"]:  # x, dy, y and dx, the weights and their gradients
        return {"bytes": 2 * (4 * T * H + 6 * H * I), "flops": 18 * T * H * I}
    return {"bytes": 2 * (2 * T * H + 3 * H * I), "flops": 6 * T * H * I}


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# ---------------------------------------------------------------------------


def _values_64(codes, scale, of_rows):
    """Codes [n, k] times their scale, one per 128 columns and per ``of_rows`` rows."""
    n, k = codes.shape
    r, c = torch.arange(n, device="cuda") // of_rows, torch.arange(k, device="cuda") // 128
    return scale.double()[r][:, c] * codes.view(torch.float8_e4m3fn).double()


def _e4m3_64(v):
    """Nearest e4m3 value of float64 ``v`` within +-448, ties to even: steps of 2^(e - 3), and of 2^-9 below 2^-6."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.clamp(torch.round(v / step) * step, -E4M3_MAX, E4M3_MAX)


def _exact_linear(s):
    w = _values_64(s["w"], s["w_scale"], 128)
    y = torch.cat([torch.einsum("tk,nk->tn", _values_64(x, f, 1), w)
                   for x, f in zip(s["x"].split(4096), s["x_scale"].split(4096))])
    return y if s["onto"] is None else y + s["onto"].double()


def _exact_shared(s):
    I = s["intermediate"]
    w13, w2 = _values_64(s["w13"], s["w13_scale"], 128), _values_64(s["w2"], s["w2_scale"], 128)
    out = []
    for x, f in zip(s["x"].split(4096), s["x_scale"].split(4096)):
        gu = torch.einsum("tk,nk->tn", _values_64(x, f, 1), w13)
        h = (gu[:, :I] / (1.0 + torch.exp(-gu[:, :I])) * gu[:, I:]).reshape(len(x), -1, 128)
        top = h.abs().max(dim=2, keepdim=True).values / E4M3_MAX
        h = (_e4m3_64(h / top.clamp(min=1e-300)) * top).reshape(len(x), I)
        out.append(torch.einsum("tk,nk->tn", h, w2))
    out = torch.cat(out)
    return out if s["onto"] is None else out + s["onto"].double()


def _exact_ffn(s):
    I, H = s["intermediate"], s["hidden"]
    w13, w2 = s["w13"].detach().double(), s["w2"].detach().double()
    gate, up = w13.split(I)
    y, dx = [], []
    dgate, dup, ddown = torch.zeros_like(gate), torch.zeros_like(up), torch.zeros_like(w2)
    for at in torch.arange(s["tokens"], device="cuda").split(4096):
        x = s["x"].detach()[at].double()
        g, u = torch.einsum("th,ih->ti", x, gate), torch.einsum("th,ih->ti", x, up)
        e = 1.0 + torch.exp(-g)
        h = g / e * u
        y.append(torch.einsum("ti,hi->th", h, w2))
        if not s["train"]:
            continue
        dy = s["dy"][at].double()
        dh = torch.einsum("th,hi->ti", dy, w2)
        du = dh * g / e
        dg = dh * u * (e + g * (e - 1.0)) / (e * e)
        dx.append(torch.einsum("ti,ih->th", dg, gate) + torch.einsum("ti,ih->th", du, up))
        dgate += torch.einsum("ti,th->ih", dg, x)
        dup += torch.einsum("ti,th->ih", du, x)
        ddown += torch.einsum("th,ti->hi", dy, h)
    out = {"y": torch.cat(y)}
    if s["train"]:
        out.update(dx=torch.cat(dx), dw13=torch.cat((dgate, dup)), dw2=ddown)
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"linear": _exact_linear, "shared": _exact_shared, "ffn": _exact_ffn}[case["op"]](s)
