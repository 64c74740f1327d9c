"""float32 outputs of the block-scaled products: the error of 32-bit sums, on every kernel."""
import pytest
import torch

import tile_gemm_amd as hts

import scaled_ref as ref
import scaled_whole as whole
from scaled_cases import SHAPES
from scaled_ref import DEV, blocks

pytestmark = pytest.mark.gpu

F32 = torch.float32


def check(y, want, off, K):
    """Each output within its error (tests/scaled_whole.py) and its own rounding, and the 2-norm within 2^-20 (growing as
    the errors do): the mean error is a quarter of the largest, 2.4e-7."""
    assert bool(((y.double() - want).abs() <= off + 2.0 ** -24 * want.abs()).all()), \
        float(((y.double() - want).abs() / (off + 2.0 ** -24 * want.abs())).max())
    assert float((y.double() - want).norm()) <= 2.0 ** -20 * max(1.0, blocks(K) / 32) ** 0.5 * float(want.norm())


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K):
    g = ref.generator(M + 3 * N + 7 * K)
    x, xs = ref.random_rows(g, M, K, pad=32, offset=16)
    w, ws = ref.random_weight(g, N, K, pad=48)
    y = hts.scaled_gemm(x, xs, hts.ScaledWeight(w, ws), out_dtype=F32)
    check(y, *whole.sums(x, xs, w, ws), K)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K", [s for s in SHAPES if s[1] * s[2] < 1.1e7])
def test_gated(M, N, K, act):
    g = ref.generator(M + 3 * N + 7 * K)
    x, xs = ref.random_rows(g, M, K, pad=16)
    wg, gs = ref.random_weight(g, N, K)
    wu, us = ref.random_weight(g, N, K, pad=16)
    h = hts.scaled_gated(x, xs, hts.ScaledWeight(wg, gs), hts.ScaledWeight(wu, us), act=act, out_dtype=F32)
    want, off = whole.gated(act, x, xs, wg, gs, wu, us)
    check(h, want, off, 4 * K)                       # (two sums and an activation: twice a sum's error)


@pytest.mark.parametrize("M,N,K", [(64, 128, 16384), (32, 333, 2064), (130, 4100, 272)])
def test_product_without_its_workspace(M, N, K):
    """The workspace that is asked for is enough for a float32 output, and none is enough too."""
    g = ref.generator(M)
    x, xs = ref.random_rows(g, M, K)
    w, ws = ref.random_weight(g, N, K)
    for nbytes in (hts.hts_scaled_gemm_workspace(M, N, K), 0):
        y = torch.empty((M, (N + 3) // 4 * 4), device=DEV)[:, :N]
        hts.scaled_gemm(x, xs, hts.ScaledWeight(w, ws), out=y, workspace=torch.empty(nbytes, dtype=torch.uint8, device=DEV))
        check(y, *whole.sums(x, xs, w, ws), K)
