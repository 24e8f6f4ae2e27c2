"""Which kernel the library makes a dense product with: the estimate of
moe_dense_host.h from the sizes, with the rates that the sources hold, so that
tests can say which form a size takes.  The library tells a plan only where K is
in parts (its workspace); test_dense_plans.py holds both together there."""

import os
import re
from typing import NamedTuple

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_ffn_route_amd", "csrc")


class Plan(NamedTuple):
    tm: int      # rows of L in a tile; 0: few_kernel
    tn: int
    splits: int  # parts of K


class Rates(NamedTuple):
    few: tuple
    narrow: float
    tile: float
    tile2: float
    wide: float
    large: float


def rates(name: str) -> Rates:
    with open(os.path.join(CSRC, name)) as f:
        text = re.search(r"constexpr Rates kRates = \{\{([^}]*)\}([^}]*)\}", f.read())
    few, rest = (tuple(float(v) for v in g.split(",") if v.strip()) for g in text.groups())
    return Rates(few, *rest)


FP8, BF16 = rates("moe_linear.hip"), rates("moe_ffn.hip")


def cdiv(a: int, b: int) -> int:
    return -(-a // b)


def few_narrow(groups: int, mt: int) -> bool:
    return groups < 200 if mt == 1 else groups <= 128


def few_blocks(blocks: int, cols: int) -> int:
    mt = cdiv(blocks, cdiv(blocks, 4))
    while mt > 1 and 2 * cols * cdiv(blocks, mt - 1) <= 256:
        mt -= 1
    return mt


def choose(m: int, n: int, kbs: int, r: Rates, few: bool, split: bool, joined: bool = False) -> Plan:
    def join(parts):
        return 3.0 + parts * m * n * 8e-6 / 6.5

    best, least = Plan(128, 128, 1), 1e30

    def offer(us, plan):
        nonlocal best, least
        if us < least:
            best, least = plan, us

    if few:
        blocks, cols = cdiv(m, 16), cdiv(n, 32)
        mt = few_blocks(blocks, cols)
        parts = cdiv(blocks, mt)
        groups = cols * parts
        if few_narrow(groups, mt):
            us = 2.8 + cdiv(2 * groups, 256) * (kbs * r.few[mt - 1] * r.narrow + 0.4)
        else:
            us = 2.8 + cdiv(groups, 256) * (kbs * r.few[mt - 1] + 0.4)
        if parts <= 65535:
            offer(us + (join(1) if joined else 0.0), Plan(0, 0, 1))
    for s in range(1, 17):
        if s > 1 and not (split and kbs >= 2 * s):
            break
        kb = cdiv(kbs, s)
        if cdiv(kbs, kb) != s:
            continue

        def per_xcd(tm, tn):
            return cdiv(cdiv(m, tm) * cdiv(n, tn), 8) * s

        t = per_xcd(128, 128)
        tail, fused = (join(s) if s > 1 else 0.0), (join(1) if joined and s == 1 else 0.0)
        offer(4.0 + (kb * r.tile if t <= 32 else cdiv(t, 64) * kb * r.tile2) + tail + fused, Plan(128, 128, s))
        offer(4.0 + cdiv(per_xcd(128, 256), 32) * kb * r.wide + tail, Plan(128, 256, s))
        offer(4.0 + cdiv(per_xcd(256, 256), 32) * kb * r.large + tail, Plan(256, 256, s))
    return best


def form(p: Plan, m: int, n: int, k_cut: bool, epilogue: str, pair: bool = False) -> str:
    """A name of the kernel and of what distinguishes its instances: few rows by
    blocks and width, tiles by stages, parts of K, a cut K-block, the epilogue."""
    parts = "parts" if p.splits > 1 else epilogue
    cut = " cut" if k_cut else ""
    if p.tm == 0:
        blocks, cols = cdiv(m, 16), cdiv(n, 32)
        mt = few_blocks(blocks, cols)
        width = "half" if few_narrow(cols * cdiv(blocks, mt), mt) else "whole"
        return f"few {mt} {width} {epilogue}{cut}"
    if p.tn == 128:
        tiles = cdiv(m, 128) * cdiv(n, 128)
        stages = 4 if cdiv(tiles, 8) * p.splits <= 32 else 2
        return f"tile {stages} {parts}{cut}"
    return f"{p.tm}x256 {parts}{cut}"


# The products of each call, as (what, form, bytes of its parts of K).

def _parts(p: Plan, m: int, pitch: int) -> int:
    return cdiv(p.splits * m * pitch * 4, 256) * 256 if p.splits > 1 else 0


def product_fp8(m: int, n: int, k: int, vec: bool = True):
    """vec: rows of out (and add) of whole 16 bytes."""
    kbs = cdiv(k, 128)
    p = Plan(0, 0, 1) if m <= 16 else choose(m, n, kbs, FP8, True, True)
    eight = vec and n % 8 == 0
    f = form(p, m, n, k % 128 != 0, "out" if p.tn != 256 or eight else "out single")
    return f, _parts(p, m, cdiv(n, 4) * 4)


def shared_expert(t: int, h: int, i: int):
    """Forms of its two products; None where at most 16 tokens take their own."""
    if t <= 16:
        return None
    first = choose(t, 2 * i, h // 128, FP8, True, True, True)
    fused = first.tn == 256 and first.splits == 1
    return form(first, t, 2 * i, False, "swiglu" if fused else "gate|up"), product_fp8(t, h, i)[0]


def shared_bytes(t: int, h: int, i: int) -> int:
    if t <= 16:
        return cdiv(t * i * 4, 256) * 256
    p = choose(t, 2 * i, h // 128, FP8, True, True, True)
    first = 0 if p.tn == 256 and p.splits == 1 else cdiv(p.splits * t * 2 * i * 4, 256) * 256
    return max(first, product_fp8(t, h, i)[1]) + cdiv(t * i, 256) * 256 + cdiv(t * (i // 128) * 4, 256) * 256


def ffn_forward(t: int, h: int, i: int):
    a, b = (choose(t, n, cdiv(k, 64), BF16, True, True) for n, k in ((2 * i, h), (h, i)))
    return ((form(a, t, 2 * i, h % 64 != 0, "swiglu"), form(b, t, h, i % 64 != 0, "out")),
            max(_parts(a, t, 2 * i), _parts(b, t, h)))


def ffn_backward(t: int, h: int, i: int, f32: bool = False):
    """Forms of dh, dx, dw13 and dw2, and the bytes of dg | du and of parts."""
    dh = choose(t, i, cdiv(h, 64), BF16, False, True)
    dx = choose(t, h, cdiv(2 * i, 64), BF16, False, True)
    w13 = choose(2 * i, h, cdiv(t, 64), BF16, False, False)
    w2 = choose(h, i, cdiv(t, 64), BF16, False, False)
    out = "f32" if f32 else "out"
    forms = (form(dh, t, i, h % 64 != 0, "dswiglu"), form(dx, t, h, 2 * i % 64 != 0, "out"),
             form(w13, 2 * i, h, t % 64 != 0, out), form(w2, h, i, t % 64 != 0, out))
    return forms, cdiv(t * 2 * i * 2, 256) * 256 + max(_parts(dh, t, i), _parts(dx, t, h))
