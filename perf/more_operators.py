"""Cases of the 8-bit linear layers: E4M3 values with a 32-bit scale for each block of 128.

  rows     a row's blocks of 128 columns to E4M3, each with its own scale
  product  Y = X W^T, X with a scale for each row and 128 columns, W with one for each 128 x 128 block
  gated    H = act(X Wg^T) * (X Wu^T) of two such weights
  mlp      a decoder block's feed-forward part: 16-bit rows to E4M3, gated, its result to E4M3, the down projection

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
        # a decode batch through a vocabulary's rows
        dict(name="product logits 24", op="product", M=24, N=32001, K=4096, pad=0, out="bf16"),
        # a chunk of a prompt beside a decode batch: too few rows for the chip, odd sizes, strided rows
        dict(name="product ragged 200", op="product", M=200, N=5000, K=5136, pad=64, out="f16"),
        # a prompt through a 7B block's down projection
        dict(name="product prefill 2048", op="product", M=2048, N=4096, K=11008, pad=0, out="bf16"),
        # a large prompt batch through one of a 13B block's inner projections
        dict(name="product prefill 8192", op="product", M=8192, N=13824, K=5120, pad=0, out="bf16"),
        # a decode batch of a 13B block
        dict(name="gated batch 48", op="gated", M=48, N=13824, K=5120, pad=0, act="gelu_tanh", out="bf16"),
        # a chunk of a prompt with a last block of 48 columns
        dict(name="gated ragged 333", op="gated", M=333, N=5504, K=4144, pad=16, act="gelu", out="f16"),
        # a single token of a 7B block
        dict(name="mlp one token", op="mlp", M=1, N=11008, K=4096, pad=0, act="silu", out="bf16"),
        # a prompt of a 7B block
        dict(name="mlp prefill 2048", op="mlp", M=2048, N=11008, K=4096, pad=0, act="silu", out="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rows", "product", "product", "gated", "mlp"])
    K = 16 * _log(rng, 4, 1024)
    pad = rng.choice([0, 0, 16, 112])
    if op == "rows":
        return dict(op=op, M=_log(rng, 1, min(16384, 16384 * 13824 // K // 2)), K=K, pad=pad,
                    dtype=rng.choice(["bf16", "f16", "f32"]))
    N = _log(rng, 64, 32768)
    if op != "product":
        N = min(13824, 16 * (N // 16))
    most = 8192 * 13824 * 5120 // (N * K * {"product": 1, "gated": 2, "mlp": 3}[op])
    case = dict(op=op, M=_log(rng, 1, max(1, min(8192, most))), N=N, K=K, pad=pad, out=rng.choice(["bf16", "f16"]))
    if op != "product":
        case["act"] = rng.choice(["silu", "silu", "gelu", "gelu_tanh"])
    return case


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
    if case["op"] in ("rows", "mlp"):
        # hidden states: each column with its own spread, a few columns far above the others
        spread = torch.exp(torch.randn(K + pad, generator=g, device=DEV))
        x = torch.randn((M, K + pad), generator=g, device=DEV) * (spread / spread.square().mean().sqrt())
        s["x"] = x.to(DT[case["dtype"] if case["op"] == "rows" else case["out"]])[:, pad // 2 // 8 * 8:][:, :K]
    else:
        s["x"] = _values(g, M, K, pad)
        # a row's scales lie one block's rows after another's, as the library writes them
        s["x_scale"] = ((torch.rand((_blocks(K), M), generator=g, device=DEV) + 0.5) * 0.01).t()
    for n in {"rows": (), "product": ("w",), "gated": ("gate", "up"), "mlp": ("gate", "up", "down")}[case["op"]]:
        rows, cols = (K, case["N"]) if n == "down" else (case["N"], K)
        s[n], s[n + "_scale"] = _weight(g, rows, cols)
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
        return {"rows": _own_rows, "product": _own_product, "gated": _own_gated, "mlp": _own_mlp}[op](s)
    return {"rows": _plain_rows, "product": _plain_product, "gated": _plain_gated, "mlp": _plain_mlp}[op](s)


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
    return dict(h=hts.scaled_gated(s["x"], s["x_scale"], s["gate_weight"], s["up_weight"], act=c["act"],
                                   out_dtype=DT[c["out"]]))


def _own_mlp(s):
    import tile_gemm_amd as hts
    return dict(y=hts.scaled_mlp(s["x"], s["gate_weight"], s["up_weight"], s["down_weight"], act=s["case"]["act"]))


def _quantized(x):
    """x [M, K] in 32 bits to E4M3 with a scale for each row and 128 columns: s = a / 448 for a block's largest
    magnitude a, values x * (448 / a).  Each of the three is rounded to 32 bits, which settles the values that lie
    between two of E4M3's."""
    M, K = x.shape
    x = torch.nn.functional.pad(x, (0, _blocks(K) * BLOCK - K)).view(M, _blocks(K), BLOCK)
    top = x.abs().amax(2).clamp_min(2.0 ** -100).double()     # (a quotient of 64 bits rounds to the 32-bit one)
    return (x * (448.0 / top).float()[:, :, None]).view(M, -1)[:, :K].to(torch.float8_e4m3fn), (top / 448.0).float()


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


def _gated32(x, s):
    g = torch.matmul(x, _weight32(s["gate"], s["gate_scale"]).t())
    u = torch.matmul(x, _weight32(s["up"], s["up_scale"]).t())
    act = s["case"]["act"]
    if act == "silu":
        return g / (1.0 + torch.exp(-g)) * u
    if act == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * 0.5 ** 0.5)) * u
    return 0.5 * g * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (g + 0.044715 * g * g * g))) * u


def _plain_gated(s):
    return dict(h=_gated32(_rows32(s["x"], s["x_scale"]), s).to(DT[s["case"]["out"]]))


def _plain_mlp(s):
    h = _gated32(_rows32(*_quantized(s["x"].float())), s)
    y = torch.matmul(_rows32(*_quantized(h)), _weight32(s["down"], s["down_scale"]).t())
    return dict(y=y.to(DT[s["case"]["out"]]))


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without, and the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def work(case):
    M, K = case["M"], case["K"]
    rows = M * K + 4 * M * _blocks(K)
    if case["op"] == "rows":
        return dict(bytes=rows + M * K * SIZE[case["dtype"]], flops=3 * M * K)
    N, weights = case["N"], {"product": 1, "gated": 2, "mlp": 3}[case["op"]]
    # an mlp reads and writes 16-bit rows of the hidden size; its inner rows need not leave the chip
    ends = 2 * M * K * SIZE[case["out"]] if case["op"] == "mlp" else rows + M * N * SIZE[case["out"]]
    return dict(bytes=ends + weights * (N * K + 4 * _blocks(N) * _blocks(K)), flops=2 * weights * M * N * K)


def _e4m3(v):
    """The nearest E4M3 value in 64 bits, ties to the even one: steps of an eighth of the power of two below, of 2^-9
    under 2^-6."""
    step = torch.exp2((torch.frexp(v)[1] - 1).clamp_min(-6).double() - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _quantized64(x):
    M, K = x.shape
    top = torch.stack([x[:, k:k + BLOCK].abs().amax(1) for k in range(0, K, BLOCK)], 1).clamp_min(2.0 ** -100)
    at = torch.arange(K, device=x.device) // BLOCK
    # the definition's own 32-bit steps: 448 / a, and its product with the value
    up = (448.0 / top).float().double()
    return dict(q=_e4m3((x * up[:, at]).float().double()), scale=top / 448.0)


def _product64(x, x_scale, w, w_scale):
    """Block by block: the values' product, then both scales."""
    y = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64, device=DEV)
    row = torch.arange(w.shape[0], device=DEV) // BLOCK
    for b in range(w_scale.shape[1]):
        k = slice(b * BLOCK, min(w.shape[1], (b + 1) * BLOCK))
        part = x[:, k].double() @ w[:, k].double().t()
        y += part * x_scale[:, b].double()[:, None] * w_scale[:, b].double()[row][None]
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rows":
        return _quantized64(s["x"].double())
    if case["op"] == "product":
        return dict(y=_product64(s["x"], s["x_scale"], s["w"], s["w_scale"]))
    x, x_scale = (s["x"], s["x_scale"]) if case["op"] == "gated" else _quantized64(s["x"].double()).values()
    g, u = _product64(x, x_scale, s["gate"], s["gate_scale"]), _product64(x, x_scale, s["up"], s["up_scale"])
    if case["act"] == "silu":
        h = g * torch.sigmoid(g) * u
    elif case["act"] == "gelu":
        h = g * torch.special.ndtr(g) * u
    else:
        h = g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)) * u
    if case["op"] == "gated":
        return dict(h=h)
    return dict(y=_product64(*_quantized64(h).values(), s["down"], s["down_scale"]))
