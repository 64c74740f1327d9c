"""Block-scaled 8-bit layers on the GPU against 64 bits (tests/scaled_ref.py says how far a result may be off)."""
import pytest
import torch

import tile_gemm_amd as hts

import scaled_ref as ref
from scaled_cases import GATED8, SHAPES
from scaled_ref import DEV, E4M3, blocks

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


# ------------------------------------------------------------------------------------------
# the quantiser
# ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("M,K,pad,dtype", [(1, 16, 0, BF16), (1, 4096, 0, F16), (3, 144, 8, F32), (64, 4096, 0, BF16),
                                           (77, 5136, 24, F16), (257, 272, 4, F32), (1000, 128, 0, BF16), (2, 16384, 0, F32)])
def test_rows_are_the_definition_bit_for_bit(M, K, pad, dtype):
    g = ref.generator(M * 7 + K)
    x = (torch.randn((M, K + 2 * pad), generator=g, device=DEV) * torch.exp(torch.randn(K + 2 * pad, generator=g, device=DEV)))
    x = x.to(dtype)[:, pad - pad % 8:][:, :K]
    q, s = hts.quantize_rows(x)
    want, scale = ref.quantized(x.double())
    assert q.shape == (M, K) and q.dtype == E4M3 and s.shape == (M, blocks(K)) and s.dtype == F32
    assert torch.equal(q.double(), want)
    assert torch.equal(s.double(), scale)


def test_rows_of_ties_zeros_and_extremes():
    # every 16-bit value once in a block whose largest magnitude is 448 * 2^k: x / scale is exact and ties are common
    bits = torch.arange(0, 65536, device=DEV, dtype=torch.int32).to(torch.int16)
    for dtype in (F16, BF16):
        x = bits.view(dtype)
        x = x[torch.isfinite(x) & (x.double().abs() < 448)].contiguous()
        x = x[: x.numel() // 127 * 127].view(-1, 127)
        x = torch.cat([x, torch.full_like(x[:, :1], 448.0)], 1)
        q, s = hts.quantize_rows(x)
        assert torch.equal(s, torch.ones_like(s))
        assert torch.equal(q.double(), ref.e4m3(x.double()))
    x = torch.zeros((5, 384), device=DEV, dtype=BF16)
    x[1, 130] = 1e-38                       # below the least top: a normal scale all the same
    x[2, 7], x[2, 8] = float("nan"), 3.0    # NaN counts for nothing and stays
    x[3, 5], x[3, 6] = float("inf"), 2.0    # an infinity: scale infinite, the rest 0
    x[4] = 1e38
    q, s = hts.quantize_rows(x)
    tiny = torch.tensor(2.0 ** -100 / 448, dtype=F32)
    assert bool((s[0] == tiny.to(DEV)).all()) and not bool(q[0].float().any())
    assert float(s[1, 1]) == float(tiny) and float(q[1, 130].float()) == 0.0
    assert float(s[2, 0]) == pytest.approx(3.0 / 448, rel=1e-7) and bool(torch.isnan(q[2, 7].float()))
    assert float(q[2, 8].float()) == 448.0
    assert float(s[3, 0]) == float("inf") and float(q[3, 6].float()) == 0.0 and bool(torch.isnan(q[3, 5].float()))
    assert bool((q[4].float() == 448).all())


@pytest.mark.parametrize("N,K,dtype", [(1, 16, BF16), (128, 128, F16), (130, 400, F32), (1000, 2064, BF16)])
def test_weight_blocks_are_the_definition_bit_for_bit(N, K, dtype):
    w = torch.randn((N, K), generator=ref.generator(N + K), device=DEV).to(dtype)
    got = hts.ScaledWeight.quantize(w)
    for r in range(blocks(N)):
        for b in range(blocks(K)):
            at = (slice(128 * r, min(N, 128 * r + 128)), slice(128 * b, min(K, 128 * b + 128)))
            part = w[at].double()
            top = part.abs().max().clamp_min(2.0 ** -100)
            assert float(got.scale[r, b]) == float((top / 448).float())
            assert torch.equal(got.values[at].double(), ref.e4m3((part * (448.0 / top).float().double()).float().double()))


# ------------------------------------------------------------------------------------------
# the product
# ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_product(M, N, K, dtype):
    g = ref.generator(M + 3 * N + 7 * K)
    x, xs = ref.random_rows(g, M, K, pad=32, offset=16)
    w, ws = ref.random_weight(g, N, K, pad=48)
    y = hts.scaled_gemm(x, xs, hts.ScaledWeight(w, ws), out_dtype=dtype)
    want, bound = ref.product(x, xs, w, ws)
    assert y.shape == (M, N) and y.dtype == dtype
    ref.check(y, want, bound, "product")


@pytest.mark.parametrize("M,N,K", [s for s in SHAPES if s[1] * s[2] < 1.1e7])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated(M, N, K, act):
    g = ref.generator(M + 3 * N + 7 * K)
    x, xs = ref.random_rows(g, M, K, pad=16)
    wg, gs = ref.random_weight(g, N, K)
    wu, us = ref.random_weight(g, N, K, pad=16)
    for dtype in (BF16, F16, F32):
        h = hts.scaled_gated(x, xs, hts.ScaledWeight(wg, gs), hts.ScaledWeight(wu, us), act=act, out_dtype=dtype)
        want, bound = ref.gated(act, x, xs, wg, gs, wu, us)
        ref.check(h, want, bound, act)


@pytest.mark.parametrize("M,N,K", GATED8)
def test_gated_rows_in_8_bits(M, N, K):
    g = ref.generator(M + 3 * N + 7 * K)
    x, xs = ref.random_rows(g, M, K)
    wg, gs = ref.random_weight(g, N, K)
    wu, us = ref.random_weight(g, N, K)
    gate, up = hts.ScaledWeight(wg, gs), hts.ScaledWeight(wu, us)
    q, s = hts.scaled_gated(x, xs, gate, up, act="silu", out_dtype=E4M3)
    want, bound = ref.gated("silu", x, xs, wg, gs, wu, us)
    at = torch.arange(N, device=DEV) // 128
    top = torch.stack([want[:, n:n + 128].abs().amax(1) for n in range(0, N, 128)], 1)
    btop = torch.stack([bound[:, n:n + 128].amax(1) for n in range(0, N, 128)], 1)
    assert s.shape == (M, blocks(N))
    # the scale: the block's largest |h| off by the block's largest bound, two roundings
    assert bool(((s.double() - top / 448).abs() <= btop / 448 + 2.0 ** -23 * top / 448).all())
    # a value: h within its bound, then half an E4M3 step (2^-4 of the value, 2^-10 at least) of the scaled value
    sc = s.double()[:, at]
    off = (q.double() * sc - want).abs()
    most = bound + sc * torch.maximum(2.0 ** -4 * ((want.abs() + bound) / sc), torch.full_like(want, 2.0 ** -10)) * (1 + 2.0 ** -20)
    assert bool((off <= most).all()), float((off / most).max())


@pytest.mark.parametrize("M,hidden,inner", [(1, 528, 1040), (8, 528, 1040), (40, 528, 1040), (300, 528, 1040)])
def test_mlp_is_its_steps(M, hidden, inner):
    g = ref.generator(M)
    x = torch.randn((M, hidden), generator=g, device=DEV).to(BF16)
    gate, up = (hts.ScaledWeight(*ref.random_weight(g, inner, hidden)) for _ in range(2))
    down = hts.ScaledWeight(*ref.random_weight(g, hidden, inner))
    y = hts.scaled_mlp(x, gate, up, down, act="gelu")
    q, s = hts.quantize_rows(x)
    h, hs = hts.scaled_gated(q, s, gate, up, act="gelu", out_dtype=E4M3)
    want, bound = ref.product(h, hs, down.values, down.scale)
    ref.check(y, want, bound, "mlp")
    x2 = x.clone()
    assert hts.scaled_mlp(x2, gate, up, down, act="gelu", out=x2) is x2
    assert torch.equal(x2, y)


@pytest.mark.parametrize("M,hidden,inner", [(1, 4096, 11008), (4, 1040, 4096), (2, 528, 2064)])
def test_the_inner_rows_of_a_few_tokens_lose_no_products(M, hidden, inner):
    """Two launches, whose inner rows are whole 32-bit sums before they become E4M3.  With sums off by 1e-7 no value is
    expected at E4M3's other neighbour (inner * M values, steps of 2^-4: 2^4 * 1e-7 of them), and what is left is the output's
    half step, 2^-11, and the second product's 2^-13 of single products, 2e-5 of its norm.  Sums that drop bits move
    ten to twenty values by an eighth of themselves: 2e-3."""
    g = ref.generator(hidden)
    x = torch.randn((M, hidden), generator=g, device=DEV).to(F16)
    gate, up = (hts.ScaledWeight(*ref.random_weight(g, inner, hidden)) for _ in range(2))
    down = hts.ScaledWeight(*ref.random_weight(g, hidden, inner))
    y = hts.scaled_mlp(x, gate, up, down)
    q, s = ref.quantized(x.double())
    h, _ = ref.gated("silu", q, s, gate.values, gate.scale, up.values, up.scale)
    want, _ = ref.product(*ref.quantized(h), down.values, down.scale)
    assert float((y.double() - want).norm() / want.norm()) < 2.0 ** -11 + 1e-4


@pytest.mark.parametrize("M,hidden,inner", [(4, 12288, 1024), (4, 1024, 12288), (3, 16384, 512), (1, 16384, 2064), (4, 12304, 1024)])
def test_a_few_tokens_of_long_rows(M, hidden, inner):
    """As many blocks of rows as a workgroup's LDS takes in two launches, and one more."""
    g = ref.generator(inner)
    x = torch.randn((M, hidden), generator=g, device=DEV).to(BF16)
    gate, up = (hts.ScaledWeight(*ref.random_weight(g, inner, hidden)) for _ in range(2))
    down = hts.ScaledWeight(*ref.random_weight(g, hidden, inner))
    y = hts.scaled_mlp(x, gate, up, down)
    q, s = ref.quantized(x.double())
    h, _ = ref.gated("silu", q, s, gate.values, gate.scale, up.values, up.scale)
    want, _ = ref.product(*ref.quantized(h), down.values, down.scale)
    # half a step of bfloat16, 2^-8, and for inner rows whose sums lose bits a few values an eighth off: 1 in 1000 of them,
    # each off by 2^-3 at most, moves the norm by 2^-3 sqrt(1e-3), 4e-3
    assert float((y.double() - want).norm() / want.norm()) < 2.0 ** -8 + 4e-3
