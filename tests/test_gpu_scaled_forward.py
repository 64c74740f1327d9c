"""block.forward on 8-bit weights: its steps are block.decode's, and its feed-forward part the definition's."""
import pytest
import torch

import tile_gemm_amd as hts
import tile_gemm_amd.block as block

import scaled_ref as ref
import scaled_whole as whole
from scaled_ref import DEV

pytestmark = pytest.mark.gpu

ALL = block.PROJECTIONS


def weights(g, hidden, inner, nq, nk, scaled, dtype):
    shape = dict(q=(nq, hidden), k=(nk, hidden), v=(nk, hidden), o=(hidden, nq), gate=(inner, hidden), up=(inner, hidden),
                 down=(hidden, inner))
    out = {}
    for n, (N, K) in shape.items():
        w = (torch.randn((N, K), generator=g, device=DEV) / K ** 0.5).to(dtype)
        out[n] = hts.ScaledWeight.quantize(w) if n in scaled else w
    return out


@pytest.mark.parametrize("scaled", [ALL, ("gate", "up", "down"), ("gate", "up"), ("gate",), ("up", "down"), ("q", "v", "o"), ()])
@pytest.mark.parametrize("M,dtype", [(1, torch.bfloat16), (37, torch.float16), (300, torch.bfloat16)])
def test_forward_is_its_steps(scaled, M, dtype):
    g = ref.generator(len(scaled) + M)
    w = weights(g, 576, 1088, 512, 256, scaled, dtype)
    x = torch.randn((M, 576), generator=g, device=DEV).to(dtype)

    def linear(v, name):
        if name in scaled:
            return hts.scaled_gemm(*hts.quantize_rows(v), w[name], out_dtype=dtype)
        return hts.dense_gemm(v, w[name])
    bufs = block.buffers(M, w, dtype, DEV)
    y = block.forward(x, w, bufs)
    assert y is bufs["down"]
    q = linear(x, "q")
    for n, want in (("q", q), ("k", linear(x, "k")), ("v", linear(x, "v")), ("o", linear(q, "o"))):
        assert torch.equal(bufs[n], want), n
    if all(n in scaled for n in ("gate", "up", "down")):
        assert torch.equal(y, hts.scaled_mlp(x, w["gate"], w["up"], w["down"]))
        whole.check_mlp(y, "silu", x, w["gate"], w["up"], w["down"])
    else:
        if "gate" in scaled and "up" in scaled:
            h = hts.scaled_gated(*hts.quantize_rows(x), w["gate"], w["up"], out_dtype=dtype)
        else:
            h = hts.silu_mul(linear(x, "gate"), linear(x, "up"))
            assert torch.equal(bufs["gate"], linear(x, "gate")) and torch.equal(bufs["up"], linear(x, "up"))
        assert torch.equal(bufs["h"], h) and torch.equal(y, linear(h, "down"))
    assert torch.equal(block.forward(x, w, block.buffers(M, w, dtype, DEV), fused=True), y)


def test_a_captured_forward_replays():
    g = ref.generator(5)
    M, dtype = 24, torch.bfloat16
    w = weights(g, 576, 1088, 512, 256, ALL, dtype)
    x = torch.zeros((M, 576), dtype=dtype, device=DEV)
    x = torch.zeros((M, 576), dtype=dtype, device=DEV)
    bufs = block.buffers(M, w, dtype, DEV)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        block.forward(x, w, bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        block.forward(x, w, bufs)
    for _ in range(3):
        new = torch.randn((M, 576), generator=g, device=DEV).to(dtype)
        x.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        got = {n: bufs[n].clone() for n in ("q", "k", "v", "o", "down")}
        again = block.buffers(M, w, dtype, DEV)
        block.forward(new, w, again)
        assert all(torch.equal(got[n], again[n]) for n in got)
