"""Block-scaled 8-bit layers as they are used: views, guards around every output, NaN around every input, workspaces, streams,
graphs, sizes past 32 bits, special values, and a decoder block on such weights."""
import pytest
import torch

import tile_gemm_amd as hts
import tile_gemm_amd.block as block

import scaled_ref as ref
from scaled_ref import DEV, E4M3, blocks

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
# M, N, K of one call for each kind of kernel: streaming, ring (three), tiles (three)
KINDS = [(3, 130, 272), (20, 3000, 400), (48, 1000, 784), (200, 1000, 1040), (700, 4000, 400), (600, 8200, 144), (1100, 4100, 144)]


def nan_rows(gen, M, K, front=16, back=48, below=3):
    """E4M3 rows inside a NaN frame: columns before and behind, rows below."""
    v, s = ref.random_rows(gen, M, K)
    frame = torch.full((M + below, front + K + back), float("nan"), device=DEV).to(E4M3)
    frame[:M, front:front + K].copy_(v)
    scales = torch.full((blocks(K) + 1, M + 5), float("nan"), device=DEV)
    scales[:-1, :M] = s.t()
    return frame[:M, front:front + K], scales[:-1, :M].t()


def nan_weight(gen, N, K):
    v, s = ref.random_weight(gen, N, K)
    frame = torch.full((N + 5, K + 32), float("nan"), device=DEV).to(E4M3)
    frame[:N, :K].copy_(v)
    scales = torch.full((blocks(N) + 1, blocks(K) + 2), float("nan"), device=DEV)
    scales[:-1, :blocks(K)] = s
    return hts.ScaledWeight(frame[:N, :K], scales[:-1, :blocks(K)])


class Guarded:
    """A [rows, cols] view inside a larger tensor; `whole()` says whether all around it is as it was."""

    def __init__(self, rows, cols, dtype, pad=16, front=16):
        lead = (front + cols + pad + 15) // 16 * 16
        self.big = torch.full((rows + 2, lead), 3.0, device=DEV).to(dtype)
        self.view = self.big[1:1 + rows, front:front + cols]

    def whole(self):
        keep = torch.ones(self.big.shape, dtype=torch.bool, device=DEV)
        off = self.view.storage_offset()
        lead = self.big.stride(0)
        r, c = off // lead, off % lead
        keep[r:r + self.view.shape[0], c:c + self.view.shape[1]] = False
        return bool((self.big.float()[keep] == 3.0).all())


@pytest.mark.parametrize("M,N,K", KINDS)
def test_nothing_outside_is_read_or_written(M, N, K):
    g = ref.generator(M + N + K)
    x, xs = nan_rows(g, M, K)
    w, u = nan_weight(g, N, K), nan_weight(g, N, K)
    y, h = Guarded(M, N, BF16), Guarded(M, N, F32)
    want, bound = ref.product(x, xs, w.values, w.scale)
    assert hts.scaled_gemm(x, xs, w, out=y.view) is y.view
    ref.check(y.view, want, bound, "product")
    hts.scaled_gated(x, xs, w, u, out=h.view)
    want, bound = ref.gated("silu", x, xs, w.values, w.scale, u.values, u.scale)
    ref.check(h.view, want, bound, "gated")
    assert y.whole() and h.whole()
    n16 = N // 16 * 16
    w, u = (hts.ScaledWeight(t.values[:n16], t.scale[:blocks(n16)]) for t in (w, u))
    q = Guarded(M, n16, E4M3)
    scales = torch.full((blocks(n16) + 2, M + 7), 3.0, device=DEV)
    hts.scaled_gated(x, xs, w, u, out=q.view, out_scale=scales[1:-1, 2:M + 2].t())
    again, s2 = hts.scaled_gated(x, xs, w, u, out_dtype=E4M3)
    assert q.whole() and torch.equal(q.view.float(), again.float()) and torch.equal(scales[1:-1, 2:M + 2].t(), s2)
    scales[1:-1, 2:M + 2] = 3.0
    assert bool((scales == 3.0).all())
    assert not bool(torch.isnan(again.float()).any())


def test_the_quantiser_stays_inside():
    x = torch.full((21, 400), float("nan"), device=DEV, dtype=BF16)
    x[:20, 8:280] = torch.randn((20, 272), generator=ref.generator(1), device=DEV).to(BF16)
    q, s = Guarded(20, 272, E4M3), torch.full((5, 24), 3.0, device=DEV)
    hts.quantize_rows(x[:20, 8:280], out=q.view, scale=s[1:4, 2:22].t())
    want, scale = ref.quantized(x[:20, 8:280].double())
    assert q.whole() and torch.equal(q.view.double(), want) and torch.equal(s[1:4, 2:22].t().double(), scale)
    s[1:4, 2:22] = 3.0
    assert bool((s == 3.0).all())


@pytest.mark.parametrize("M,N,K", KINDS)
def test_special_values_stay_in_their_row(M, N, K):
    g = ref.generator(M + N)
    x, xs = ref.random_rows(g, M, K)
    xs = xs.t().contiguous().t()
    w = hts.ScaledWeight(*ref.random_weight(g, N, K))
    clean = hts.scaled_gemm(x, xs, w, out_dtype=F32)
    x = x.clone()
    x.view(torch.uint8)[1, K - 1] = 0x7F            # NaN
    xs[2 % M, blocks(K) - 1] = float("inf")
    w.values.view(torch.uint8)[N // 2, 0] = 0xFF    # NaN of the other sign
    y = hts.scaled_gemm(x, xs, w, out_dtype=F32)
    assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[2]).any()) and bool(torch.isnan(y[:, N // 2]).all())
    keep = torch.ones(M, N, dtype=torch.bool, device=DEV)
    keep[1:3] = False
    keep[:, N // 2] = False
    assert torch.equal(y[keep], clean[keep])
    # rows of zeros, whatever their scales
    z = torch.zeros_like(x)
    assert not bool(hts.scaled_gemm(z, ref.random_rows(g, M, K)[1], hts.ScaledWeight(*ref.random_weight(g, N, K))).any())


def test_largest_and_smallest_values():
    # every value +-448 or 2^-9: sums of 128 * 448^2 and of 128 * 2^-18 are exact in 32 bits
    for v in (448.0, 2.0 ** -9):
        sign = torch.where(torch.rand((40, 384), generator=ref.generator(5), device=DEV) < 0.5, -1.0, 1.0)
        x, w = (sign * v).to(E4M3), (sign.flip(0) * v).to(E4M3)
        one = torch.ones((3, 40), device=DEV)
        y = hts.scaled_gemm(x, one.t(), hts.ScaledWeight(w, torch.ones((1, 3), device=DEV)), out_dtype=F32)
        assert torch.equal(y.double(), x.double() @ w.double().t())


@pytest.mark.parametrize("M,N,K", KINDS + [(64, 128, 16384)])
def test_workspaces(M, N, K):
    """A split product runs unsplit without its workspace; E4M3 rows that need theirs are refused without it."""
    g = ref.generator(M)
    x, xs = ref.random_rows(g, M, K)
    n16 = N // 16 * 16
    w, u = (hts.ScaledWeight(*ref.random_weight(g, n16, K)) for _ in range(2))
    want, bound = ref.product(x, xs, w.values, w.scale)
    for nbytes in (0, 16, hts.hts_scaled_gemm_workspace(M, n16, K)):
        y = torch.empty((M, n16), dtype=BF16, device=DEV)
        hts.scaled_gemm(x, xs, w, out=y, workspace=torch.empty(nbytes, dtype=torch.uint8, device=DEV))
        ref.check(y, want, bound, f"product, {nbytes} bytes")
    need = hts.hts_scaled_gated_workspace(M, n16, K, E4M3)
    full, scale = hts.scaled_gated(x, xs, w, u, out_dtype=E4M3)
    short = torch.empty(max(0, need - 16), dtype=torch.uint8, device=DEV)
    try:
        q, s = hts.scaled_gated(x, xs, w, u, out_dtype=E4M3, workspace=short)
        assert torch.equal(q.float(), full.float()) and torch.equal(s, scale)
    except hts.HTSError as e:
        assert e.status == 6 and need > 0
    with pytest.raises(hts.HTSError) as e:
        hts.scaled_mlp(torch.zeros((M, K), dtype=BF16, device=DEV), w, u, hts.ScaledWeight(*ref.random_weight(g, K, n16)),
                       workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 6


def test_no_rows():
    w = hts.ScaledWeight(*ref.random_weight(ref.generator(0), 48, 32))
    x, s = hts.quantize_rows(torch.empty((0, 32), dtype=BF16, device=DEV))
    assert x.shape == (0, 32) and s.shape == (0, 1)
    assert hts.scaled_gemm(x, s, w).shape == (0, 48)
    assert hts.scaled_gated(x, s, w, w).shape == (0, 48)
    q, s2 = hts.scaled_gated(x, s, w, w, out_dtype=E4M3)
    assert q.shape == (0, 48) and s2.shape == (0, 1)
    d = hts.ScaledWeight(*ref.random_weight(ref.generator(0), 32, 48))
    assert hts.scaled_mlp(torch.empty((0, 32), dtype=F16, device=DEV), w, w, d).shape == (0, 32)


@pytest.mark.parametrize("M,N,K", KINDS + [(64, 128, 16384)])
def test_the_same_bits_again(M, N, K):
    g = ref.generator(N)
    x, xs = ref.random_rows(g, M, K)
    w, u = (hts.ScaledWeight(*ref.random_weight(g, N // 16 * 16, K)) for _ in range(2))
    a = [hts.scaled_gemm(x, xs, w, out_dtype=F32), *hts.scaled_gated(x, xs, w, u, out_dtype=E4M3)]
    for _ in range(3):
        b = [hts.scaled_gemm(x, xs, w, out_dtype=F32), *hts.scaled_gated(x, xs, w, u, out_dtype=E4M3)]
        assert all(torch.equal(p.float(), q.float()) for p, q in zip(a, b))


def test_rows_do_not_depend_on_their_batch():
    """A row alone and in a batch of the same kernel: the same bits."""
    g = ref.generator(9)
    x, xs = ref.random_rows(g, 300, 400)
    w = hts.ScaledWeight(*ref.random_weight(g, 1000, 400))
    y = hts.scaled_gemm(x, xs, w, out_dtype=F32)
    z = hts.scaled_gemm(x.flip(0).contiguous(), xs.flip(0).t().contiguous().t(), w, out_dtype=F32)
    assert torch.equal(y, z.flip(0))


def test_two_streams_at_once():
    g = ref.generator(3)
    M, N, K = 64, 128, 16384                       # split: each call needs a workspace of its own
    jobs = []
    for _ in range(2):
        x, xs = ref.random_rows(g, M, K)
        w = hts.ScaledWeight(*ref.random_weight(g, N, K))
        jobs.append((x, xs, w, hts.scaled_gemm(x, xs, w)))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [hts.scaled_gemm(x, xs, w, stream=s) for (x, xs, w, _), s in zip(jobs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(y, j[3]) for y, j in zip(got, jobs))


@pytest.mark.parametrize("M", [1, 4, 20, 70, 300])
def test_a_captured_mlp_replays(M):
    hidden, inner = 400, 1040
    g = ref.generator(M)
    gate, up = (hts.ScaledWeight(*ref.random_weight(g, inner, hidden)) for _ in range(2))
    down = hts.ScaledWeight(*ref.random_weight(g, hidden, inner))
    square = hts.ScaledWeight(down.values[:, :hidden], down.scale[:, :blocks(hidden)])
    x, out = torch.zeros((M, hidden), dtype=F16, device=DEV), torch.zeros((M, hidden), dtype=F16, device=DEV)
    space = torch.empty(hts.hts_scaled_mlp_workspace(M, hidden, inner), dtype=torch.uint8, device=DEV)
    y32 = torch.zeros((M, hidden), dtype=F32, device=DEV)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        hts.scaled_mlp(x, gate, up, down, out=out, workspace=space)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        hts.scaled_mlp(x, gate, up, down, out=out, workspace=space)
        q, s = hts.quantize_rows(out)
        hts.scaled_gemm(q, s, square, out=y32)
    for k in range(4):
        new = torch.randn((M, hidden), generator=g, device=DEV).to(F16)
        x.copy_(new)
        space.fill_(255)                           # (nothing of the last replay's workspace is used)
        graph.replay()
        torch.cuda.synchronize()
        want = hts.scaled_mlp(new, gate, up, down)
        assert torch.equal(out, want)
        q2, s2 = hts.quantize_rows(want)
        assert torch.equal(y32, hts.scaled_gemm(q2, s2, square, out_dtype=F32))


def test_offsets_past_32_bits():
    g = ref.generator(2)
    # outputs: 70,000 x 33,000 elements; the last rows and columns are right
    M, N, K = 70_000, 33_000, 16
    x, xs = ref.random_rows(g, M, K)
    w = hts.ScaledWeight(*ref.random_weight(g, N, K))
    y = hts.scaled_gemm(x, xs, w)
    at = torch.tensor([0, 1, 32_767, 65_080, 69_998, 69_999], device=DEV)
    want, bound = ref.product(x.view(torch.uint8)[at].view(E4M3), xs[at], w.values, w.scale)
    ref.check(y[at], want, bound, "far outputs")
    del y
    # rows 4,080 bytes apart: the last ones lie past 2^31 bytes
    M, N, K, ld = 600_000, 40, 32, 4080
    big = torch.zeros((M, ld), dtype=torch.uint8, device=DEV).view(E4M3)
    x, xs = ref.random_rows(g, M, K)
    big[:, :K].copy_(x)
    w = hts.ScaledWeight(*ref.random_weight(g, N, K))
    y = hts.scaled_gemm(big[:, :K], xs, w)
    want, bound = ref.product(x.view(torch.uint8)[-50:].view(E4M3), xs[-50:], w.values, w.scale)
    ref.check(y[-50:], want, bound, "far rows")
    # the same as a weight, streamed and not
    far = hts.ScaledWeight(big[:, :K], (torch.rand((blocks(M), 1), generator=g, device=DEV) + 0.5) * 0.01)
    for rows in (2, 40):
        v, vs = ref.random_rows(g, rows, K)
        y = hts.scaled_gemm(v, vs, far)
        want, bound = ref.product(v, vs, x.view(torch.uint8)[-64:].view(E4M3), far.scale[-1:])
        ref.check(y[:, -64:], want, bound, "far weights")       # (600,000 is 64 past a multiple of 128)
    # the quantiser: 2^31 elements and more
    x = torch.zeros((300_000, 8192), dtype=F16, device=DEV)
    x[-3:] = torch.randn((3, 8192), generator=g, device=DEV).to(F16)
    q, s = hts.quantize_rows(x)
    want, scale = ref.quantized(x[-3:].double())
    assert torch.equal(q[-3:].double(), want) and torch.equal(s[-3:].double(), scale)


# ------------------------------------------------------------------------------------------
# a decoder block
# ------------------------------------------------------------------------------------------

def _block_weights(g, hidden, inner, nq, nk, scaled, dtype):
    shape = dict(q=(nq, hidden), k=(nk, hidden), v=(nk, hidden), o=(hidden, nq), gate=(inner, hidden), up=(inner, hidden),
                 down=(hidden, inner))
    out = {}
    for n, (N, K) in shape.items():
        w = (torch.randn((N, K), generator=g, device=DEV) / K ** 0.5).to(dtype)
        out[n] = hts.ScaledWeight.quantize(w) if n in scaled else w
    return out


ALL = ("q", "k", "v", "o", "gate", "up", "down")


@pytest.mark.parametrize("scaled", [ALL, ("gate", "up", "down"), ("gate", "up"), ("up",), ("q", "o", "down"), ()])
def test_a_block_decodes_as_its_steps(scaled):
    """block.decode on any mixture of 8-bit and 16-bit weights against the public steps, one by one, bit for bit (each is
    tested against 64 bits by itself), over three tokens with a captured last one."""
    dtype, B, hidden, inner, heads, kv, dim, page = BF16, 5, 512, 1024, 4, 2, 128, 16
    g = ref.generator(len(scaled))
    w = _block_weights(g, hidden, inner, heads * dim, kv * dim, scaled, dtype)
    norms = [hts.Norm("rms", (1 + 0.1 * torch.randn(hidden, generator=g, device=DEV)).to(dtype)) for _ in range(2)]
    plan = hts.rope_plan(dim)

    def fresh():
        cache = hts.kv_cache(12, page, kv, dim, dtype)
        table = torch.full((B, 2), -1, dtype=torch.int32, device=DEV)
        return cache, table, torch.arange(12, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)

    def by_steps(x, cache, table, step):
        r, y = hts.residual_norm(x, None, pre=norms[0])

        def linear(v, name):
            if name in scaled:
                return hts.scaled_gemm(*hts.quantize_rows(v), w[name], out_dtype=dtype)
            return hts.dense_gemm(v, w[name])
        q, k, v = (linear(y, n) for n in "qkv")
        hts.rope_cache(q, k, v, step.positions, step.slots, plan, cache, starts=step.starts)
        o = linear(hts.paged_attn(q, cache, table, step.lengths), "o")
        r, y = hts.residual_norm(o, r, pre=norms[1])
        if all(n in scaled for n in ("gate", "up", "down")):
            return hts.scaled_mlp(y, w["gate"], w["up"], w["down"]), r
        if "gate" in scaled and "up" in scaled:
            h = hts.scaled_gated(*hts.quantize_rows(y), w["gate"], w["up"], out_dtype=dtype)
        else:
            h = hts.silu_mul(linear(y, "gate"), linear(y, "up"))
        return linear(h, "down"), r

    ones = torch.ones(B, dtype=torch.int32, device=DEV)
    a, b = fresh(), fresh()
    layer = block.Layer(w, a[0], *norms)
    head_a = head_b = None
    cached_a, cached_b = a[3], b[3]
    for _ in range(3):
        x = torch.randn((B, hidden), generator=g, device=DEV).to(dtype)
        sa = hts.kv_step(cached_a, ones, a[2], a[1], page, B, free_head=head_a)
        sb = hts.kv_step(cached_b, ones, b[2], b[1], page, B, free_head=head_b)
        got, want = block.decode(x, None, layer, sa, a[1], plan), by_steps(x, b[0], b[1], sb)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert torch.equal(a[0].k, b[0].k) and torch.equal(a[0].v, b[0].v) and bool(torch.isfinite(got[0]).all())
        cached_a, head_a, cached_b, head_b = sa.lengths, sa.head, sb.lengths, sb.head
    # the last token once more, captured (its cache entries are the same)
    x2, bufs = x.clone(), block.buffers(B, w, dtype, DEV)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        block.decode(x2, None, layer, sa, a[1], plan, bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out, _ = block.decode(x2, None, layer, sa, a[1], plan, bufs)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got[0])


def test_a_block_refuses_shapes_that_do_not_fit():
    g = ref.generator(4)
    w = _block_weights(g, 512, 1024, 512, 256, ALL, BF16)
    cache = hts.kv_cache(4, 16, 2, 128, BF16)
    n = hts.Norm("rms")
    layer = block.Layer(w, cache, n, n)
    assert layer.dtype is None and block.kept_flops(1, w) == 2.0 * sum(t.N * t.K for t in w.values())
    with pytest.raises(hts.HTSError):
        block.Layer(dict(w, down=w["up"]), cache, n, n)
    mixed = dict(w, o=torch.zeros((512, 512), dtype=F16, device=DEV))
    assert block.Layer(mixed, cache, n, n).dtype == F16
    with pytest.raises(hts.HTSError):
        block.Layer(dict(mixed, q=torch.zeros((512, 512), dtype=BF16, device=DEV)), cache, n, n)
    with pytest.raises(hts.HTSError):
        block.Layer(dict(w, q=torch.zeros((512, 512), device=DEV).to(E4M3)), cache, n, n)


def test_helpers_refuse():
    g = ref.generator(6)
    x, xs = ref.random_rows(g, 8, 256)
    w = hts.ScaledWeight(*ref.random_weight(g, 48, 256))
    bad = [
        lambda: hts.quantize_rows(x),                                              # already 8 bits
        lambda: hts.quantize_rows(torch.zeros((4, 24), device=DEV)),               # K not a multiple of 16
        lambda: hts.quantize_rows(torch.zeros((4, 32))),                           # not on a GPU
        lambda: hts.quantize_rows(torch.zeros((32, 32), device=DEV).t()[:, :16]),  # not along its rows
        lambda: hts.ScaledWeight(w.values, w.scale[:, :1]),
        lambda: hts.ScaledWeight(w.values.float(), w.scale),
        lambda: hts.ScaledWeight(w.values[:, :200], w.scale),                      # 200 columns
        lambda: hts.ScaledWeight(w.values, w.scale.double()),
        lambda: hts.scaled_gemm(x[:, :128], xs, w),
        lambda: hts.scaled_gemm(x, xs[:4], w),
        lambda: hts.scaled_gemm(x, xs.contiguous(), w),                            # scales row by row
        lambda: hts.scaled_gemm(x.float(), xs, w),
        lambda: hts.scaled_gemm(x, xs, w, out_dtype=E4M3),
        lambda: hts.scaled_gemm(x, xs, w, out=torch.empty((8, 47), device=DEV)),
        lambda: hts.scaled_gemm(x, xs, w, out=torch.empty((8, 50), device=DEV)[:, :48]),     # ldy = 50
        lambda: hts.scaled_gated(x, xs, w, hts.ScaledWeight(*ref.random_weight(g, 64, 256))),
        lambda: hts.scaled_gated(x, xs, w, w, act="relu"),
        lambda: hts.scaled_gated(x, xs, w, w, out_scale=xs),
        lambda: hts.scaled_gated(x, xs, *[hts.ScaledWeight(*ref.random_weight(g, 40, 256))] * 2, out_dtype=E4M3),   # 40 % 16
        lambda: hts.scaled_mlp(x, w, w, w),
        lambda: hts.scaled_mlp(torch.zeros((8, 256), dtype=BF16, device=DEV), w, w, w),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(hts.HTSError):
            call()
            pytest.fail(f"call {n} went through")
    torch.cuda.synchronize()
