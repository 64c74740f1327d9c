"""Rows that become E4M3 in 64 bits: which values a 32-bit sum decides.

A sum of K products in 32 bits is off by a few roundings of 2^-24 of its partial sums.  With s the root of the sum of
the products' squares (the size of a partial sum), K / 128 scaled blocks add up with errors of 2^-24 / sqrt(3) s each, half of
them at that size: sqrt(K / 256) * 0.58 * 2^-24 s, and as much again inside the blocks, 2.4e-7 s for K = 4096.  2^-20 (s +
|sum|) is four to six times that, so that none of ten million sums is expected outside; it grows with the root of K
beyond 4096.  The 8-bit instruction's sums are off by 1.5e-5 s, sixteen times as much.

A value whose distance from an E4M3 tie is larger than its error has one right neighbour.  One that is nearer
(about one in ten thousand) may lie a step away, and what it moves is added up.
"""
import torch

import scaled_ref as ref
from scaled_ref import blocks


def _rows(x, xs):
    return x.double() * ref.spread(xs, *x.shape, False)


def sums(x, xs, w, ws):
    """(sums, their errors) in 64 bits."""
    X, W = _rows(x, xs), w.double() * ref.spread(ws, *w.shape, True)
    y = X @ W.t()
    size = (X.square() @ W.square().t()).sqrt()
    return y, 2.0 ** -20 * max(1.0, blocks(x.shape[1]) / 32) ** 0.5 * (size + y.abs())


def gated(name, x, xs, wg, gs, wu, us):
    """(H, error): the activation is off by a few 2^-24 of itself, where it cancels of its argument."""
    g, eg = sums(x, xs, wg, gs)
    u, eu = sums(x, xs, wu, us)
    a = ref.act(name, g)
    ea = ref.SLOPE * eg + 2.0 ** -21 * (a.abs() + g.abs())
    return a * u, a.abs() * eu + ea * u.abs() + 2.0 ** -23 * (a * u).abs()


def rows(h, e):
    """(values, scale, relative error of the scale, undecided, step): h to E4M3.  step: of a value, in the values' units."""
    N = h.shape[1]
    q, scale = ref.quantized(h)
    at = torch.arange(N, device=h.device) // 128
    parts = [slice(n, min(N, n + 128)) for n in range(0, N, 128)]
    top = torch.stack([h[:, p].abs().amax(1) for p in parts], 1).clamp_min(2.0 ** -100)
    off = torch.stack([e[:, p].amax(1) for p in parts], 1) / top
    v = h.abs() * (448.0 / top)[:, at]
    dv = e * (448.0 / top)[:, at] + v * (off[:, at] + 2.0 ** -22)
    step = torch.exp2((torch.frexp(v)[1] - 1).clamp_min(-6).double() - 3.0)
    tie = ((v / step) - torch.floor(v / step) - 0.5).abs() * step
    return q, scale, off + 2.0 ** -22, tie <= dv, step


def check_rows(q, s, h, e):
    """E4M3 rows q with scales s against h (64 bits, off by e): decided values are the definition's, others a step off at most."""
    want, scale, off, undecided, step = rows(h, e)
    assert bool(((s.double() - scale).abs() <= off * scale).all()), float(((s.double() - scale).abs() / (off * scale)).max())
    got = q.double()
    wrong = (got != want) & ~undecided
    assert not bool(wrong.any()), f"{int(wrong.sum())} of {wrong.numel()} values are not the definition's ({int(undecided.sum())} undecided)"
    assert bool(((got - want).abs() <= 1.001 * step).all())      # (a tie's two neighbours are a step apart)
    return undecided


def mlp(act, x, gate, up, down):
    """(Y, for each row what undecided values may move its 2-norm by) of a feed-forward part, in 64 bits."""
    q, s = ref.quantized(x.double())
    h, e = gated(act, q, s, gate.values, gate.scale, up.values, up.scale)
    hq, hs, off, undecided, step = rows(h, e)
    W = down.values.double() * ref.spread(down.scale, *down.shape, True)
    at = torch.arange(h.shape[1], device=h.device) // 128
    y = (hq * hs[:, at]) @ W.t()
    return y, ((undecided * step * hs[:, at]) @ W.square().sum(0).sqrt()) + off.amax(1) * y.norm(dim=1)


def check_mlp(got, act, x, gate, up, down):
    """Row by row: the output's rounding (what rounding the exact row costs, whose square over N outputs varies by
    1 / sqrt(N) or so: four times that), the second product's instruction (1.5e-5 of the norm, twice that), and what the
    undecided values move."""
    want, moved = mlp(act, x, gate, up, down)
    rounding = (want.to(got.dtype).double() - want).norm(dim=1)
    most = rounding * (1 + 4 / want.shape[1] ** 0.5) + 3e-5 * want.norm(dim=1) + moved
    off = (got.double() - want).norm(dim=1)
    assert bool((off <= most).all()), \
        f"{int((off > most).sum())} of {off.numel()} rows off, worst {float((off / most).max()):.3g} of its bound"
