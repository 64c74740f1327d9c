"""Whole sums as they are used: offsets past 32 bits, special values inside E4M3 rows, two feed-forward parts at once, replays."""
import pytest
import torch

import tile_gemm_amd as hts

import scaled_ref as ref
import scaled_whole as whole
from scaled_ref import DEV, E4M3, blocks

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def test_outputs_past_32_bits():
    g = ref.generator(2)
    M, N, K = 70_000, 33_008, 16
    x, xs = ref.random_rows(g, M, K)
    w, ws = ref.random_weight(g, N, K)
    u, us = ref.random_weight(g, N, K)
    gate, up = hts.ScaledWeight(w, ws), hts.ScaledWeight(u, us)
    at = torch.tensor([0, 1, 32_767, 65_058, 65_059, 69_998, 69_999], device=DEV)      # 2^31 bytes end in row 65,059
    some, scales = x.view(torch.uint8)[at].view(E4M3), xs[at]
    q, s = hts.scaled_gated(x, xs, gate, up, out_dtype=E4M3)
    whole.check_rows(q.view(torch.uint8)[at].view(E4M3), s[at], *whole.gated("silu", some, scales, w, ws, u, us))
    del q, s
    y = hts.scaled_gemm(x, xs, gate, out_dtype=F32)
    want, off = whole.sums(some, scales, w, ws)
    ref.check(y[at], want, off, "32-bit outputs")


# one size for each way to E4M3 rows: streaming, rings in one part and more, tiles with parts, tiles that make the rows
WAYS = [(3, 4112, 400), (16, 1408, 4096), (48, 1408, 1040), (64, 1408, 4096), (100, 11008, 4096), (700, 4000, 400), (500, 4112, 1040)]


@pytest.mark.parametrize("M,N,K", WAYS)
def test_special_values_in_e4m3_rows(M, N, K):
    """NaN in a row of X or an infinite scale: that row alone.  NaN in a weight's row whose outputs are zero otherwise: that
    column, and neither the scales nor the other values of its block."""
    g = ref.generator(M + N)
    x, xs = ref.random_rows(g, M, K)
    xs = xs.t().contiguous().t()
    (w, ws), (u, us) = ref.random_weight(g, N, K), ref.random_weight(g, N, K)
    column = N // 2 + 5
    u = u.clone()
    u.view(torch.uint8)[column] = 0
    gate = hts.ScaledWeight(w, ws)
    q, s = hts.scaled_gated(x, xs, gate, hts.ScaledWeight(u, us), out_dtype=E4M3)
    assert not bool(q[:, column].float().any())
    x, bad = x.clone(), u.clone()
    x.view(torch.uint8)[1, K - 1] = 0x7F
    xs[2, blocks(K) - 1] = float("inf")
    bad.view(torch.uint8)[column, 0] = 0xFF
    q2, s2 = hts.scaled_gated(x, xs, gate, hts.ScaledWeight(bad, us), out_dtype=E4M3)
    assert bool(torch.isnan(q2[1].float()).all()) and bool(torch.isnan(q2[:, column].float()).all())
    assert not bool((torch.isfinite(q2[2].float()) & torch.isfinite(s2[2].repeat_interleave(128)[:N]) & (q2[2].float() != 0)).any())
    rows = torch.ones(M, dtype=torch.bool, device=DEV)
    rows[1:3] = False
    cols = torch.ones(N, dtype=torch.bool, device=DEV)
    cols[column] = False
    assert torch.equal(q2.float()[rows][:, cols], q.float()[rows][:, cols]) and torch.equal(s2[rows], s[rows])


def test_rows_of_zeros_and_of_one_value():
    """A block of zeros has the smallest scale; every value of a block alike becomes 448 each."""
    for M, N, K in WAYS:
        g = ref.generator(N)
        x = torch.zeros((M, K), device=DEV).to(E4M3)
        one = torch.ones((blocks(K), M), device=DEV).t()
        gate = torch.ones((N, K), device=DEV).to(E4M3)
        weight = hts.ScaledWeight(gate, torch.full((blocks(N), blocks(K)), 1.0 / K, device=DEV))
        q, s = hts.scaled_gated(x, one, weight, weight, out_dtype=E4M3)
        assert not bool(q.float().any()) and bool((s == torch.tensor(2.0 ** -100, device=DEV) / 448).all())
        x = torch.ones((M, K), device=DEV).to(E4M3)
        q, s = hts.scaled_gated(x, one, weight, weight, out_dtype=E4M3)
        assert bool((q.float() == 448).all()) and bool(((s.double() * 448 - 0.7310585786).abs() < 1e-6).all())


@pytest.mark.parametrize("M,hidden,inner", [(2, 400, 1040), (24, 1040, 1408), (300, 528, 4112)])
def test_two_feed_forward_parts_at_once(M, hidden, inner):
    """On two streams, each with its own workspace, over and over: the results of calls one by one."""
    g = ref.generator(M)
    jobs = []
    for _ in range(2):
        gate, up = (hts.ScaledWeight(*ref.random_weight(g, inner, hidden)) for _ in range(2))
        down = hts.ScaledWeight(*ref.random_weight(g, hidden, inner))
        x = torch.randn((M, hidden), generator=g, device=DEV).to(F16)
        jobs.append((x, gate, up, down, hts.scaled_mlp(x, gate, up, down)))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [hts.scaled_mlp(*j[:4], stream=s) for j, s in zip(jobs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(y, j[4]) for y, j in zip(got, jobs))


@pytest.mark.parametrize("M,N,K", WAYS)
def test_captured_rows_replay(M, N, K):
    g = ref.generator(K)
    x, xs = ref.random_rows(g, M, K)
    gate, up = (hts.ScaledWeight(*ref.random_weight(g, N, K)) for _ in range(2))
    fixed, scale = x.clone(), xs.t().contiguous().t()
    out, out_scale = torch.empty((M, N), dtype=E4M3, device=DEV), torch.empty((blocks(N), M), device=DEV).t()
    y = torch.empty((M, (N + 3) // 4 * 4), device=DEV)[:, :N]
    space = torch.empty(max(16, hts.hts_scaled_gated_workspace(M, N, K, E4M3), hts.hts_scaled_gemm_workspace(M, N, K)), dtype=torch.uint8,
                        device=DEV)

    def calls():
        hts.scaled_gated(fixed, scale, gate, up, out=out, out_scale=out_scale, workspace=space)
        hts.scaled_gemm(fixed, scale, gate, out=y, workspace=space)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        calls()
    for _ in range(4):
        new, new_scale = ref.random_rows(g, M, K)
        fixed.view(torch.uint8).copy_(new.view(torch.uint8))
        scale.copy_(new_scale)
        space.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        q, s = hts.scaled_gated(new, new_scale, gate, up, out_dtype=E4M3)
        assert torch.equal(out.float(), q.float()) and torch.equal(out_scale, s)
        assert torch.equal(y, hts.scaled_gemm(new, new_scale, gate, out_dtype=F32))
