"""Rows that become E4M3, and feed-forward parts, against 64 bits value by value (tests/scaled_whole.py)."""
import pytest
import torch

import tile_gemm_amd as hts

import scaled_ref as ref
import scaled_whole as whole
from scaled_ref import DEV, E4M3, blocks
from scaled_whole_cases import E4M3_ROWS

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("M,N,K", E4M3_ROWS)
def test_gated_rows_are_the_definitions_values(M, N, K):
    g = ref.generator(M + 3 * N + 7 * K)
    x, xs = ref.random_rows(g, M, K, pad=16)
    wg, gs = ref.random_weight(g, N, K)
    wu, us = ref.random_weight(g, N, K)
    q, s = hts.scaled_gated(x, xs, hts.ScaledWeight(wg, gs), hts.ScaledWeight(wu, us), act="silu", out_dtype=E4M3)
    assert q.shape == (M, N) and s.shape == (M, blocks(N))
    h, e = whole.gated("silu", x, xs, wg, gs, wu, us)
    undecided = whole.check_rows(q, s, h, e)
    assert int(undecided.sum()) <= 8 + M * N // 500             # (else the comparison would say little)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K", [(3, 272, 400), (48, 1040, 784), (300, 1040, 528), (1100, 1424, 272)])
def test_gated_rows_of_the_other_activations(M, N, K, act):
    g = ref.generator(M + N)
    x, xs = ref.random_rows(g, M, K)
    wg, gs = ref.random_weight(g, N, K)
    wu, us = ref.random_weight(g, N, K, pad=16)
    q, s = hts.scaled_gated(x, xs, hts.ScaledWeight(wg, gs), hts.ScaledWeight(wu, us), act=act, out_dtype=E4M3)
    whole.check_rows(q, s, *whole.gated(act, x, xs, wg, gs, wu, us))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M", [1, 2, 5, 16, 48, 128, 300, 2048])
@pytest.mark.parametrize("hidden,inner", [(4096, 11008), (5120, 13824), (528, 1040)])
def test_a_feed_forward_part_is_its_definition(hidden, inner, M, dtype):
    g = ref.generator(M + hidden)
    x = torch.randn((M, hidden), generator=g, device=DEV).to(dtype)
    gate, up = (hts.ScaledWeight(*ref.random_weight(g, inner, hidden)) for _ in range(2))
    down = hts.ScaledWeight(*ref.random_weight(g, hidden, inner))
    y = hts.scaled_mlp(x, gate, up, down)
    assert y.dtype == dtype
    whole.check_mlp(y, "silu", x, gate, up, down)
