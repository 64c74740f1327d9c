"""Block-scaled 8-bit layers in 64 bits, from their definitions, and how far a result may be off.

An element's error has three sources.  (1) The 8-bit matrix instruction keeps, in each group of eight products along K, 13
bits below the power of two of the largest one and drops the rest of each product: at most 8 * 2^-13 of the largest
product in a group, and that is at most the product of the group's largest |x| and largest |w|.  (2) Sums of 32 bits: a
block's sum takes at most 16 additions of groups, the scale product, its multiplication and one addition for each block
follow, each off by 2^-24 of a partial sum, which the sum of |x| |w| bounds.  (3) The output's rounding, half a step.
"""
import torch

DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


def blocks(n):
    return -(-n // 128)


def e4m3(v):
    """Nearest E4M3 value in 64 bits, ties to even, no saturation needed below 464."""
    step = torch.exp2((torch.frexp(v)[1] - 1).clamp_min(-6).double() - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def quantized(x):
    """(values, scale) in 64 bits of rows x (64 bits), with the definition's own 32-bit steps."""
    K = x.shape[1]
    top = torch.stack([x[:, k:k + 128].abs().amax(1) for k in range(0, K, 128)], 1).clamp_min(2.0 ** -100)
    up = (448.0 / top).float().double()
    at = torch.arange(K, device=x.device) // 128
    return e4m3((x * up[:, at]).float().double()), (top / 448.0).float().double()


def spread(scale, rows, cols, row_block):
    s = scale.double()
    if row_block:
        s = s.repeat_interleave(128, 0)[:rows]
    return s.repeat_interleave(128, 1)[:, :cols]


def product(x, xs, w, ws):
    """(Y, bound on the error of its 32-bit sums) in 64 bits."""
    (M, K), N = x.shape, w.shape[0]
    X, W = x.double() * spread(xs, M, K, False), w.double() * spread(ws, N, K, True)
    y = X @ W.t()
    pad = (-K) % 8
    assert pad == 0

    def tops(v):
        return v.abs().view(v.shape[0], -1, 8).amax(2)
    dropped = 8 * 2.0 ** -13 * (tops(X) @ tops(W).t())
    sums = (16 + 3 + blocks(K)) * 2.0 ** -24 * (X.abs() @ W.abs().t())
    return y, dropped + sums


def act(name, g):
    if name == "silu":
        return g * torch.sigmoid(g)
    if name == "gelu":
        return g * torch.special.ndtr(g)
    return g * torch.sigmoid(2.0 * (2.0 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3))


# the largest slope of each activation (silu 1.0998, gelu 1.1289, its tanh form 1.1290), rounded up
SLOPE = 1.13


def gated(name, x, xs, wg, gs, wu, us):
    """(H, bound) in 64 bits.  The activation is 32-bit: g, e^-g (2 units), a sum, a quotient and the products are each off
    by a few 2^-24; 16 of them cover all three forms, relative to |act(g)| + 2^-24 |g| where a form cancels."""
    g, eg = product(x, xs, wg, gs)
    u, eu = product(x, xs, wu, us)
    a = act(name, g)
    ea = SLOPE * eg + 16 * 2.0 ** -24 * (a.abs() + g.abs() * 2.0 ** -1)
    return a * u, a.abs() * eu + ea * u.abs() + ea * eu + 2.0 ** -23 * (a * u).abs()


def random_rows(gen, M, K, pad=0, offset=0):
    """E4M3 rows over the whole range of the type, rows `pad` apart, and block-major scales."""
    v = (torch.randn((M, K + pad), generator=gen, device=DEV) * 100).clamp_(-448, 448).to(E4M3)[:, offset:offset + K]
    s = ((torch.rand((blocks(K), M), generator=gen, device=DEV) + 0.5) * 0.01).t()
    return v, s


def random_weight(gen, N, K, pad=0):
    v = (torch.randn((N, K + pad), generator=gen, device=DEV) * 100).clamp_(-448, 448).to(E4M3)[:, :K]
    s = (torch.rand((blocks(N), blocks(K)), generator=gen, device=DEV) + 0.5) * (0.01 / K ** 0.5)
    return v, s


def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def check(got, want, bound, what):
    """Every element within the bound and half a step of its type (for E4M3's neighbour see the callers)."""
    eps = torch.finfo(got.dtype).eps / 2
    off = (got.double() - want).abs()
    # 2^-24: the smallest half step of binary16's subnormals is 2^-25
    most = bound + eps * (want.abs() + bound) + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    assert bool((off <= most).all()), f"{what}: {int((off > most).sum())} of {off.numel()} off, worst {float((off / most).max()):.3g} of the bound"
