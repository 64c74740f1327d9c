"""Cases of the 8-bit linear layers: E4M3 values with a 32-bit scale for each block of 128.

  rows     a row's blocks of 128 columns to E4M3, each with its own scale
  product  Y = X W^T, X with a scale for each row and 128 columns, W with one for each 128 x 128 block
  gated    H = act(X Wg^T) * (X Wu^T) of two such weights, in 16 or 32 bits or as E4M3 rows with scales

``run`` computes an operator in elementary torch operations (values times scales, 32-bit products and sums), or, with
``own`` set, calls the library.  Shapes are those of the 7B / 13B layers the repository measures (hidden 4096 / 5120,
inner 11008 / 13824) or generic ones.
"""
import math

import torch

own = False

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "fp8": 1}
BLOCK = 128


def listed():
    return [
        # the rows of a decode batch before its projections; latency
        dict(name="rows decode 64", op="rows", M=64, K=4096, pad=0, dtype="bf16"),
        # a ragged batch whose last block holds 16 columns, read from the middle of wider rows
        dict(name="rows ragged 777", op="rows", M=777, K=5136, pad=48, dtype="f16"),
        # a large prompt batch in front of a 13B block's down projection
        dict(name="rows prefill 16384", op="rows", M=16384, K=13824, pad=0, dtype="bf16"),
        # a single chat's token through a 7B block's output projection: the smallest product
        dict(name="product one token", op="product", M=1, N=4096, K=4096, pad=0, out="bf16"),
        # a decode batch through a vocabulary's rows, logits in 32 bits for sampling
        dict(name="product logits 24", op="product", M=24, N=32001, K=4096, pad=0, out="f32"),
        # a chunk of a prompt beside a decode batch: too few rows for the chip, odd sizes, strided rows
        dict(name="product ragged 200", op="product", M=200, N=5000, K=5136, pad=64, out="f16"),
        # a prompt through a 7B block's down projection
        dict(name="product prefill 2048", op="product", M=2048, N=4096, K=11008, pad=0, out="bf16"),
        # a large prompt batch through one of a 13B block's inner projections
        dict(name="product prefill 8192", op="product", M=8192, N=13824, K=5120, pad=0, out="bf16"),
        # a single token of a 7B block, ready for the down projection
        dict(name="gated one token", op="gated", M=1, N=11008, K=4096, pad=0, act="silu", out="fp8"),
        # a decode batch of a 13B block
        dict(name="gated batch 48", op="gated", M=48, N=13824, K=5120, pad=0, act="gelu_tanh", out="bf16"),
        # a chunk of a prompt with a last block of 48 columns
        dict(name="gated ragged 333", op="gated", M=333, N=5504, K=4144, pad=16, act="gelu", out="f16"),
        # a prompt of a 7B block, ready for the down projection
        dict(name="gated prefill 2048", op="gated", M=2048, N=11008, K=4096, pad=0, act="silu", out="fp8"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rows", "product", "product", "gated"])
    K = 16 * _log(rng, 4, 1024)
    pad = rng.choice([0, 0, 16, 112])
    if op == "rows":
        return dict(op=op, M=_log(rng, 1, min(16384, 16384 * 13824 // K // 2)), K=K, pad=pad,
                    dtype=rng.choice(["bf16", "f16", "f32"]))
    N = _log(rng, 64, 32768)
    if op == "gated":
        N = min(13824, 16 * (N // 16))
    most = 8192 * 13824 * 5120 // (N * K * (2 if op == "gated" else 1))
    M = _log(rng, 1, max(1, min(8192, most)))
    if op == "product":
        return dict(op=op, M=M, N=N, K=K, pad=pad, out=rng.choice(["bf16", "f16", "f32"]))
    return dict(op=op, M=M, N=N, K=K, pad=pad, act=rng.choice(["silu", "silu", "gelu", "gelu_tanh"]),
                out=rng.choice(["bf16", "f16", "fp8", "fp8"]))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _blocks(n):
    return -(-n // BLOCK)


def _values(g, rows, cols, pad):
    """E4M3 values spread over the type's range, rows `pad` bytes apart."""
    v = torch.randn((rows, cols + pad), generator=g, device=DEV) * 100.0
    return v.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)[:, :cols]


def _weight(g, N, K):
    """A weight of unit gain: values near 100, scales near 1 / 100 sqrt(K)."""
    scale = (torch.rand((_blocks(N), _blocks(K)), generator=g, device=DEV) + 0.5) * (0.01 / math.sqrt(K))
    return _values(g, N, K, 0), scale


def prepare(case, seed):
    g = _gen(seed)
    M, K, pad = case["M"], case["K"], case["pad"]
    s = dict(case=case)
    if case["op"] == "rows":
        # hidden states: each column with its own spread, a few columns far above the others
        spread = torch.exp(torch.randn(K + pad, generator=g, device=DEV))
        x = torch.randn((M, K + pad), generator=g, device=DEV) * spread
        s["x"] = x.to(DT[case["dtype"]])[:, pad // 2 // 8 * 8:][:, :K]
        return s
    s["x"] = _values(g, M, K, pad)
    # a row's scales lie one block's rows after another's, as the library writes them
    s["x_scale"] = ((torch.rand((_blocks(K), M), generator=g, device=DEV) + 0.5) * 0.01).t()
    names = ("w",) if case["op"] == "product" else ("gate", "up")
    for n in names:
        s[n], s[n + "_scale"] = _weight(g, case["N"], K)
        if own:
            import tile_gemm_amd as hts
            s[n + "_weight"] = hts.ScaledWeight(s[n], s[n + "_scale"])
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"rows": _own_rows, "product": _own_product, "gated": _own_gated}[op](s)
    return {"rows": _plain_rows, "product": _plain_product, "gated": _plain_gated}[op](s)


def _own_rows(s):
    import tile_gemm_amd as hts
    q, scale = hts.quantize_rows(s["x"])
    return dict(q=q, scale=scale)


def _own_product(s):
    import tile_gemm_amd as hts
    return dict(y=hts.scaled_gemm(s["x"], s["x_scale"], s["w_weight"], out_dtype=DT[s["case"]["out"]]))


def _own_gated(s):
    import tile_gemm_amd as hts
    c = s["case"]
    got = hts.scaled_gated(s["x"], s["x_scale"], s["gate_weight"], s["up_weight"], act=c["act"], out_dtype=DT[c["out"]])
    return dict(q=got[0], scale=got[1]) if c["out"] == "fp8" else dict(h=got)


def _quantized(x):
    """x [M, K] in 32 bits to E4M3 with a scale for each row and 128 columns."""
    M, K = x.shape
    x = torch.nn.functional.pad(x, (0, _blocks(K) * BLOCK - K)).view(M, _blocks(K), BLOCK)
    scale = x.abs().amax(2).clamp_min(2.0 ** -100) / 448.0
    return (x / scale[:, :, None]).view(M, -1)[:, :K].to(torch.float8_e4m3fn), scale


def _plain_rows(s):
    q, scale = _quantized(s["x"].float())
    return dict(q=q, scale=scale)


def _rows32(x, scale):
    return x.float() * scale.repeat_interleave(BLOCK, 1)[:, :x.shape[1]]


def _weight32(w, scale):
    N, K = w.shape
    return w.float() * scale.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


def _plain_product(s):
    y = torch.matmul(_rows32(s["x"], s["x_scale"]), _weight32(s["w"], s["w_scale"]).t())
    return dict(y=y.to(DT[s["case"]["out"]]))


def _plain_gated(s):
    c = s["case"]
    x = _rows32(s["x"], s["x_scale"])
    g = torch.matmul(x, _weight32(s["gate"], s["gate_scale"]).t())
    u = torch.matmul(x, _weight32(s["up"], s["up_scale"]).t())
    if c["act"] == "silu":
        h = g / (1.0 + torch.exp(-g)) * u
    elif c["act"] == "gelu":
        h = 0.5 * g * (1.0 + torch.erf(g * 0.5 ** 0.5)) * u
    else:
        h = 0.5 * g * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (g + 0.044715 * g * g * g))) * u
    if c["out"] == "fp8":
        q, scale = _quantized(h)
        return dict(q=q, scale=scale)
    return dict(h=h.to(DT[c["out"]]))


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without, and the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def work(case):
    M, K = case["M"], case["K"]
    rows = M * K + 4 * M * _blocks(K)
    if case["op"] == "rows":
        return dict(bytes=rows + M * K * SIZE[case["dtype"]], flops=3 * M * K)
    N, weights = case["N"], 2 if case["op"] == "gated" else 1
    out = M * N * SIZE[case["out"]] + (4 * M * _blocks(N) if case["out"] == "fp8" else 0)
    return dict(bytes=rows + weights * (N * K + 4 * _blocks(N) * _blocks(K)) + out, flops=2 * weights * M * N * K)


def _e4m3(v):
    """The nearest E4M3 value in 64 bits, ties to the even one: steps of an eighth of the power of two below, of 2^-9
    under 2^-6."""
    step = torch.exp2((torch.frexp(v)[1] - 1).clamp_min(-6).double() - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _quantized64(x):
    M, K = x.shape
    scale = torch.stack([x[:, k:k + BLOCK].abs().amax(1) for k in range(0, K, BLOCK)], 1).clamp_min(2.0 ** -100) / 448.0
    at = torch.arange(K, device=x.device) // BLOCK
    return dict(q=_e4m3(x / scale[:, at]), scale=scale)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rows":
        return _quantized64(s["x"].double())

    def product(w, w_scale):
        # block by block: the whole numbers' product, then both scales
        y = torch.zeros((case["M"], case["N"]), dtype=torch.float64, device=DEV)
        row = torch.arange(case["N"], device=DEV) // BLOCK
        for b in range(_blocks(case["K"])):
            k = slice(b * BLOCK, min(case["K"], (b + 1) * BLOCK))
            part = s["x"][:, k].double() @ w[:, k].double().t()
            y += part * s["x_scale"][:, b].double()[:, None] * w_scale[:, b].double()[row][None]
        return y

    if case["op"] == "product":
        return dict(y=product(s["w"], s["w_scale"]))
    g, u = product(s["gate"], s["gate_scale"]), product(s["up"], s["up_scale"])
    if case["act"] == "silu":
        h = g * torch.sigmoid(g) * u
    elif case["act"] == "gelu":
        h = g * torch.special.ndtr(g) * u
    else:
        h = g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)) * u
    return _quantized64(h) if case["out"] == "fp8" else dict(h=h)
