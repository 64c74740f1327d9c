"""Plain 64-bit forms of the steps around the products, for the parity tests (numpy, no GPU code)."""
import math

import numpy as np

EPS = {"f16": 2.0 ** -10, "bf16": 2.0 ** -7, "f32": 2.0 ** -23}   # torch.finfo(t).eps; a rounding is off by half of it
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}   # half the smallest subnormal


def kv_step(cached, added, page, free, head, table, width, tokens):
    """(table, lengths, starts, slots, positions, head) of hts_kv_step, in Python integers."""
    top = 2 ** 31 - 1
    table = [list(r) for r in table]
    head = max(head, 0)
    lengths, starts, slots, positions, total = [], [0], [], [], 0
    cap = width * page
    for b, (c, a) in enumerate(zip(cached, added)):
        c, a = max(c, 0), max(a, 0)
        n = min(c + a, cap)
        for j in range(-(-min(c, cap) // page), -(-n // page)):
            table[b][j] = free[head] if head < len(free) else -1
            head += 1
        for p in range(c, c + a):
            if len(slots) == tokens:
                break
            held = table[b][p // page] if p < cap else -1
            slots.append(held * page + p % page if held >= 0 else -1)
            positions.append(min(p, top))
        lengths.append(min(n, top))
        total += a
        starts.append(min(total, top))
    pad = [-1] * (tokens - len(slots))
    return table, lengths, starts, slots + pad, positions + pad, min(head, top)


def rope_turns(rot, theta=10000.0, rule="plain", factor=1.0, context=0.0, low=1.0, high=32.0):
    """Turns per position in extended precision (80 bits on x86)."""
    L = np.longdouble
    i = np.arange(rot // 2).astype(L)
    two_pi = 2 * L("3.14159265358979323846264338327950288")
    base = L(theta) * L(factor) ** (L(rot) / (rot - 2)) if rule == "base" else L(theta)
    f = base ** (-2 * i / L(rot))
    if rule == "linear":
        f = f / L(factor)
    if rule == "ramp":
        c = np.clip((L(context) * f / two_pi - L(low)) / (L(high) - L(low)), 0, 1)
        f = f * (c + (1 - c) / L(factor))
    if rule == "ramp_pairs":
        def pair(n):
            return rot * math.log(context / (2 * math.pi * n)) / (2 * math.log(theta))
        first = min(max(math.floor(pair(high)), 0), rot - 1)
        last = min(max(math.ceil(pair(low)), 0), rot - 1)
        c = np.clip(1 - (i - first) / L(max(last - first, 1e-3)), 0, 1)
        f = f * (c + (1 - c) / L(factor))
    return f / two_pi


def rope(x, positions, turns, dim, layout, magnitude):
    """x [T, heads*dim] float64 -> rotated, and |x| + |y| of each entry's pair (0 for copied entries)."""
    T = x.shape[0]
    rot = 2 * len(turns)
    x = x.reshape(T, -1, dim)
    angle = positions.astype(np.longdouble)[:, None] * turns[None]
    angle = (angle - np.floor(angle)) * 2 * np.longdouble("3.14159265358979323846264338327950288")
    c, s = np.cos(angle).astype(np.float64)[:, None], np.sin(angle).astype(np.float64)[:, None]
    out, size = x.copy(), np.zeros_like(x)
    ia = np.arange(rot // 2) if layout == "half" else np.arange(0, rot, 2)
    ib = ia + (rot // 2 if layout == "half" else 1)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = magnitude * (a * c - b * s), magnitude * (a * s + b * c)
    size[..., ia] = size[..., ib] = abs(magnitude) * (np.abs(a) + np.abs(b))
    return out.reshape(T, -1), size.reshape(T, -1)


def attn(q, k, v, table, lengths, page, scale, window, hk):
    """q [B, heads, dim], k and v [pages, page, hk, dim] float64 -> out, lse, and for each output entry a bound
    on its error but for the last rounding (32-bit scores and sums, weights held to 2^-16 of their value)."""
    B, heads, dim = q.shape
    out, lse, err = np.zeros_like(q), np.full((B, heads), -np.inf), np.zeros_like(q)
    lse_err = np.zeros((B, heads))
    group = heads // hk
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * page)
        t = np.arange(max(0, n - window) if window else 0, n)
        ids = table[b, t // page]
        ok = (ids >= 0) & (ids < k.shape[0])
        t, ids = t[ok], ids[ok]
        if not len(t):
            continue
        for h in range(heads):
            kk, vv = k[ids, t % page, h // group], v[ids, t % page, h // group]
            s = kk @ q[b, h] * scale
            # a sum of dim products in 32 bits, scaled: at most (dim + 4) roundings of its absolute terms
            ds = (dim + 4) * 2.0 ** -24 * abs(scale) * np.max(np.abs(kk) @ np.abs(q[b, h]))
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            out[b, h], lse[b, h] = p @ vv / l, m + math.log(l)
            # the exponent's argument is rounded too: |s - m| 2^-23, where e^(s-m) still counts (below 2^5)
            rel = 2 * ds + 2.0 ** -18
            err[b, h] = (rel + 2.0 ** -16 + len(t) * 2.0 ** -24) * (p @ np.abs(vv)) / l
            lse_err[b, h] = ds + 2.0 ** -18 + len(t) * 2.0 ** -24 + 2.0 ** -22 * abs(lse[b, h])
    return out, lse, err, lse_err


SUM = 2.0 ** -18   # a 32-bit sum of a row: up to 32 terms in a thread, then a tree of at most 10 levels, and the
#                    roundings of the norm's own multiplications: under 64 half steps of 2^-24


def norm(x, e, kind, eps, w, b):
    """norm(x) * w + b over rows in 64 bits, and a bound on the 32-bit form's error from inputs off by at most e."""
    w = np.ones(x.shape[1]) if w is None else w
    b = np.zeros(x.shape[1]) if b is None else b
    if kind == "none":
        return x, e
    centred = x
    if kind == "layer":
        centred = x - x.mean(1, keepdims=True)
        e = e + e.mean(1, keepdims=True) + SUM * (np.abs(x) + np.abs(x).mean(1, keepdims=True))
    r = 1 / np.sqrt((centred ** 2).mean(1, keepdims=True) + eps)
    y = centred * r * w
    # r's relative error: half the mean square's, at most rms(e) * r plus the sum's own
    rel = np.sqrt((e ** 2).mean(1, keepdims=True)) * r + SUM
    return y + b, np.abs(w) * r * e + np.abs(y) * rel + SUM * (np.abs(y) + np.abs(b))


def residual_norm(block, residual, post, pre, gate, act, scale):
    """post and pre: (kind, eps, weight, bias).  -> r, bound, y, bound (float64, no rounding)."""
    if block is None:
        x, e = 0.0, 0.0
    else:
        x, e = norm(block, np.zeros_like(block), *post)
        if gate is not None:
            g = gate if act == "none" else 1 / (1 + np.exp(-gate)) * (gate if act == "silu" else 1.0)
            x, e = x * g, e * np.abs(g) + 2.0 ** -20 * np.abs(x * g)
        x, e = scale * x, abs(scale) * e + 2.0 ** -23 * np.abs(scale * x)
    r = x + (0.0 if residual is None else residual)
    e = e + 2.0 ** -23 * np.abs(r)
    y, ey = norm(r, e, *pre)
    return r, e, y, ey
