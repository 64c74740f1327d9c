"""The steps around the products together: a two-layer model of hybrid tile-sparse blocks generating token by
token over a paged cache that grows (block.decode and kv_step), against the same model in 64 bits over the whole
history, and captured in one graph whose replays advance their own state."""
import numpy as np
import pytest
import torch

import serving_ref as ref
import tile_gemm_amd as hts
import tile_gemm_amd.block as block
from helpers import DEV, say

pytestmark = pytest.mark.gpu
HID, INNER, HQ, HK, DIM, PAGE = 512, 1024, 4, 2, 128, 16


class Model:
    def __init__(self, cache_dtype, seed=0, pages=64, post=True):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)

        def rand(*shape, sigma=1.0, mean=0.0):
            return (torch.randn(shape, generator=g, device=DEV) * sigma + mean).bfloat16()
        rows = dict(q=HQ * DIM, k=HK * DIM, v=HK * DIM, o=HID, gate=INNER, up=INNER, down=HID)
        cols = dict(o=HQ * DIM, down=INNER)
        rng = np.random.default_rng(seed)
        self.layers, self.dense = [], []
        for i in range(2):
            w, d = {}, {}
            for name, n in rows.items():
                k = cols.get(name, HID)
                W = rand(n, k, sigma=k ** -0.5)
                m = (rng.random((n // 128) * (k // 128)) < 0.5).astype(np.uint8)
                w[name] = hts.pack(W, m, 128, 128)
                d[name] = hts.unpack(w[name]).double().cpu().numpy()
            scales = [None, None]
            if cache_dtype == torch.float8_e4m3fn:
                scales = [torch.full((HK,), s, device=DEV) for s in (0.05, 0.02)]
            cache = hts.kv_cache(pages, PAGE, HK, DIM, cache_dtype, DEV, "head" if i else "token", *scales)
            norm = lambda: hts.Norm("rms", rand(HID, sigma=0.1, mean=1.0), eps=1e-5)  # noqa: E731
            self.layers.append(block.Layer(w, cache, norm(), norm(), norm() if post else None, norm() if post else None,
                                           attn_gate=rand(HID, sigma=0.1, mean=0.8) if post else None,
                                           residual_scale=0.7 if post else 1.0, window=0 if i else 24))
            self.dense.append(d)
        self.final = hts.Norm("rms", rand(HID, sigma=0.1, mean=1.0), eps=1e-5)
        self.plan = hts.rope_plan(DIM, 64, layout="interleaved", device=DEV)

    def forward(self, x, step, table):
        r = None
        for layer in self.layers:
            x, r = block.decode(x, r, layer, step, table, self.plan)
        return hts.residual_norm(x, r, pre=self.final, keep_residual=False)[1]

    def reference(self, xs):
        """The model in 64 bits over one request's inputs xs [T, HID]; returns the output of every position."""
        def norm(x, n):
            return x if n is None else x / np.sqrt((x ** 2).mean(1, keepdims=True) + n.eps) * n.weight.double().cpu().numpy()
        T, turns, r = len(xs), ref.rope_turns(64), xs
        for layer, w in zip(self.layers, self.dense):
            y = norm(r, layer.input_norm)
            q, k, v = (y @ w[n].T for n in "qkv")
            pos = np.arange(T)
            q = ref.rope(q, pos, turns, DIM, "interleaved", 1.0)[0].reshape(T, HQ, DIM)
            k = ref.rope(k, pos, turns, DIM, "interleaved", 1.0)[0].reshape(T, HK, DIM)
            v = v.reshape(T, HK, DIM)
            a = np.zeros((T, HQ, DIM))
            for t in range(T):
                lo = max(0, t + 1 - layer.window) if layer.window else 0
                for h in range(HQ):
                    s = k[lo:t + 1, h // 2] @ q[t, h] * DIM ** -0.5
                    p = np.exp(s - s.max())
                    a[t, h] = p @ v[lo:t + 1, h // 2] / p.sum()
            gate = 1.0 if layer.attn_gate is None else layer.attn_gate.double().cpu().numpy()
            r = r + layer.residual_scale * gate * norm(a.reshape(T, -1) @ w["o"].T, layer.post_attn_norm)
            y = norm(r, layer.mlp_norm)
            g = y @ w["gate"].T
            h = g / (1 + np.exp(-g)) * (y @ w["up"].T)
            r = r + layer.residual_scale * norm(h @ w["down"].T, layer.post_mlp_norm)
        return norm(r, self.final)


def _run(model, xs, steps, active, capacity, graph=False):
    """Generate `steps` tokens for `active` requests in a batch of `capacity` rows; outputs [steps, capacity, HID]."""
    width = 8
    free = torch.randperm(64, device=DEV).int()
    table = torch.full((capacity, width), -1, dtype=torch.int32, device=DEV)
    cached = torch.zeros(capacity, dtype=torch.int32, device=DEV)
    added = torch.zeros(capacity, dtype=torch.int32, device=DEV)
    added[:active] = 1
    head = torch.zeros(1, dtype=torch.int32, device=DEV)
    x = torch.zeros((capacity, HID), dtype=torch.bfloat16, device=DEV)

    def step():
        st = hts.kv_step(cached, added, free, table, PAGE, capacity, free_head=head)
        y = model.forward(x, st, table)
        cached.copy_(st.lengths)
        head.copy_(st.head)
        return y
    outs = []
    if graph:
        keep = [t.clone() for layer in model.layers for t in (layer.cache.k.view(torch.uint8), layer.cache.v.view(torch.uint8))]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            y = step()
        # the warm-up's state is taken back: its tokens, its pages and the caches
        cached.zero_()
        head.zero_()
        table.fill_(-1)
        for layer, k, v in zip(model.layers, keep[::2], keep[1::2]):
            layer.cache.k.view(torch.uint8).copy_(k)
            layer.cache.v.view(torch.uint8).copy_(v)
    for i in range(steps):
        x[:active] = xs[i]
        if graph:
            gr.replay()
            torch.cuda.synchronize()
            junk = (x.float() * 2).sum()               # eager work between the replays
            assert torch.isfinite(junk)
        else:
            y = step()
        outs.append(y.clone())
    return torch.stack(outs), cached, head, table


@pytest.mark.parametrize("cache_dtype", [torch.bfloat16, torch.float8_e4m3fn], ids=["bf16", "fp8"])
@pytest.mark.parametrize("post", [True, False])
def test_generation_matches_the_model_in_64_bits(cache_dtype, post):
    model = Model(cache_dtype, post=post)
    B, steps = 3, 37                                     # three pages of 16, past the window of 24
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    xs = torch.randn((steps, B, HID), generator=g, device=DEV).bfloat16()
    y, cached, head, table = _run(model, xs, steps, B, B)
    assert cached.tolist() == [steps] * B and int(head) == 3 * B
    got = y.double().cpu().numpy()
    for b in range(B):
        want = model.reference(xs[:, b].double().cpu().numpy())
        err = np.linalg.norm(got[:, b] - want, axis=1) / np.linalg.norm(want, axis=1)
        say(f"[decode] {cache_dtype} post={post} request {b}: relative error {err.max():.4f}")
        # every block rounds 12 vectors to 16 bits, each to at most 2^-9 of its length on average (half a step of 2^-8,
        # uniform), and every stage carries relative errors on about as they are: 24 * 2^-9 if they all added up.
        # An 8-bit cache rounds k and v once more, to 2^-4 / sqrt(3) each, in two blocks; k's goes into the scores
        # (of deviation about 1), v's averages over the tokens: at most half of each reaches the block's output.
        assert err.max() <= 24 * 2.0 ** -9 + (4 * 0.5 * 2.0 ** -4 / 3 ** 0.5 if cache_dtype != torch.bfloat16 else 0.0)


@pytest.mark.parametrize("cache_dtype", [torch.bfloat16, torch.float8_e4m3fn], ids=["bf16", "fp8"])
def test_blocks_attend_to_what_their_cache_holds(cache_dtype):
    # each block's cache and output product in its own step, so that a scale or a window that is wrong in one of them
    # shows: the cache against k and v in 64 bits, the product against 64-bit attention over that cache
    model = Model(cache_dtype, seed=12, post=False)
    B, steps = 3, 40
    g = torch.Generator(device=DEV)
    g.manual_seed(13)
    free, table = torch.randperm(64, generator=g, device=DEV).int(), torch.full((B, 8), -1, dtype=torch.int32, device=DEV)
    cached, ones, head = torch.zeros(B, dtype=torch.int32, device=DEV), torch.ones(B, dtype=torch.int32, device=DEV), None
    for t in range(steps):
        x, r = torch.randn((B, HID), generator=g, device=DEV).bfloat16(), None
        st = hts.kv_step(cached, ones, free, table, PAGE, B, free_head=head)
        for n, (layer, w) in enumerate(zip(model.layers, model.dense)):
            bufs = block.buffers(B, layer.weights, torch.bfloat16, DEV)
            stream = x.double() if r is None else (r.float() + x.float()).double()
            x, r = block.decode(x, r, layer, st, table, model.plan, bufs)
            if t not in (0, steps - 1):
                continue
            c = layer.cache
            ks, vs = ((1.0, 1.0) if c.k_scale is None else (s.double().cpu().numpy()[:, None] for s in (c.k_scale, c.v_scale)))
            kc, vc = c.k.float().double().cpu().numpy() * ks, c.v.float().double().cpu().numpy() * vs
            tab, weight = table.cpu().numpy(), layer.input_norm.weight.double()
            y = (stream / torch.sqrt((stream ** 2).mean(1, keepdim=True) + 1e-5) * weight).cpu().numpy()
            at = np.arange(max(0, t + 1 - layer.window) if layer.window else 0, t + 1)
            for b in range(B):
                k, v = y[b] @ w["k"].T, y[b] @ w["v"].T
                k = ref.rope(k[None], np.array([t]), ref.rope_turns(64), DIM, "interleaved", 1.0)[0]
                ids = tab[b, at // PAGE]
                for want, held, s, m in ((k.reshape(HK, DIM), kc, ks, w["k"]), (v.reshape(HK, DIM), vc, vs, w["v"])):
                    got = held[ids[-1], t % PAGE]
                    # half steps of 2^-8: y's through the product (its largest gain), k or v after it, k turned; then the
                    # cache's: the same, or 2^-4 of the value and 2^-10 among the small ones
                    tol = 2.0 ** -8 * (np.linalg.norm(m, 2) * np.linalg.norm(y[b]) + 2 * np.linalg.norm(want))
                    if cache_dtype != torch.bfloat16:
                        tol += 2.0 ** -4 * np.linalg.norm(want) + 2.0 ** -10 * np.max(s) * want.size ** 0.5
                    assert np.linalg.norm(got - want) <= tol, (n, t, b)
                q = bufs["q"][b].double().cpu().numpy().reshape(HQ, DIM)
                a = np.zeros((HQ, DIM))
                for h in range(HQ):
                    sc = kc[ids, at % PAGE, h // 2] @ q[h] * DIM ** -0.5
                    p = np.exp(sc - sc.max())
                    a[h] = p @ vc[ids, at % PAGE, h // 2] / p.sum()
                want, got = w["o"] @ a.reshape(-1), bufs["o"][b].double().cpu().numpy()
                # attention rounded once (through the product's largest gain), the product once, and 32-bit sums
                tol = 2.0 ** -8 * (np.linalg.norm(w["o"], 2) * np.linalg.norm(a) + np.linalg.norm(want)) * (1 + 2.0 ** -6)
                say(f"[decode] {cache_dtype} layer {n} step {t} request {b}: {np.linalg.norm(got - want):.2e} of {tol:.2e}")
                assert np.linalg.norm(got - want) <= tol
        cached, head = st.lengths, st.head


def test_generation_on_row_major_weights():
    # the same blocks on the unpacked weights: the same products up to the order of their sums
    model = Model(torch.bfloat16, seed=4)
    g = torch.Generator(device=DEV)
    g.manual_seed(11)
    xs = torch.randn((5, 2, HID), generator=g, device=DEV).bfloat16()
    for layer in model.layers:
        layer.weights = {n: hts.unpack(w) for n, w in layer.weights.items()}
    y = _run(model, xs, 5, 2, 2)[0].double().cpu().numpy()
    for b in range(2):
        want = model.reference(xs[:, b].double().cpu().numpy())
        assert np.all(np.linalg.norm(y[:, b] - want, axis=1) <= 24 * 2.0 ** -9 * np.linalg.norm(want, axis=1))


def test_generation_in_a_graph():
    # one captured step, replayed: page growth, slots and lengths advance on the device; a batch of 3 in 5 rows
    model = Model(torch.bfloat16, seed=1)
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    xs = torch.randn((35, 3, HID), generator=g, device=DEV).bfloat16()
    torch.manual_seed(3)
    eager, c0, h0, t0 = _run(model, xs, 35, 3, 5)
    for layer in model.layers:
        layer.cache.k.zero_()
        layer.cache.v.zero_()
    torch.manual_seed(3)
    replayed, c1, h1, t1 = _run(model, xs, 35, 3, 5, graph=True)
    assert torch.equal(eager[:, :3], replayed[:, :3])
    assert c0.tolist() == c1.tolist() == [35, 35, 35, 0, 0] and int(h0) == int(h1) == 9 and torch.equal(t0, t1)
    assert bool(torch.isfinite(replayed).all())


def test_padding_rows_change_nothing():
    # the same requests in a batch with and without padding rows behind them
    model = Model(torch.bfloat16, seed=2)
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    xs = torch.randn((20, 4, HID), generator=g, device=DEV).bfloat16()
    torch.manual_seed(5)
    a, _, _, ta = _run(model, xs, 20, 4, 4)
    k0 = [layer.cache.k.clone() for layer in model.layers]
    for layer in model.layers:
        layer.cache.k.zero_()
        layer.cache.v.zero_()
    torch.manual_seed(5)
    b, _, _, tb = _run(model, xs, 20, 4, 9)
    assert torch.equal(a, b[:, :4]) and torch.equal(ta, tb[:4])
    for k, layer in zip(k0, model.layers):
        assert torch.equal(k, layer.cache.k)


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_paused_requests(graph):
    # requests that add no token in some steps, in the middle of the batch: each one's outputs are those of its own tokens
    model = Model(torch.bfloat16, seed=5)
    B, steps, width = 5, 24, 4
    active = np.random.default_rng(1).random((steps, B)) < 0.6
    active[0], active[1], active[:, 3] = True, [1, 0, 1, 0, 1], False       # request 3 has no token at all
    g = torch.Generator(device=DEV)
    g.manual_seed(10)
    xs = torch.randn((steps, B, HID), generator=g, device=DEV).bfloat16()
    free = torch.arange(64, device=DEV).int()
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    cached, added, head = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (B, B, 1))
    x = torch.zeros((B, HID), dtype=torch.bfloat16, device=DEV)

    def step():
        st = hts.kv_step(cached, added, free, table, PAGE, B, free_head=head)
        y = model.forward(x, st, table)
        cached.copy_(st.lengths)
        head.copy_(st.head)
        return y
    if graph:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()                                       # nothing is added
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            y = step()
    outs = []
    for i in range(steps):
        x.copy_(xs[i])
        added.copy_(torch.from_numpy(active[i].astype(np.int32)))
        if graph:
            gr.replay()
            torch.cuda.synchronize()
        else:
            y = step()
        outs.append(y.clone())
    got = torch.stack(outs).double().cpu().numpy()
    assert cached.tolist() == active.sum(0).tolist()
    for b in (0, 1, 2, 4):
        mine = active[:, b]
        want = model.reference(xs[:, b].double().cpu().numpy()[mine])
        err = np.linalg.norm(got[mine, b] - want, axis=1) / np.linalg.norm(want, axis=1)
        say(f"[decode] paused, request {b} of {mine.sum()} tokens: relative error {err.max():.4f}")
        assert err.max() <= 24 * 2.0 ** -9               # as in test_generation_matches_the_model_in_64_bits


def test_a_request_that_adds_two_tokens_is_not_decoded_silently():
    model = Model(torch.bfloat16, seed=5)
    free, table = torch.arange(64, device=DEV).int(), torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    cached, added = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 0, 0], [1, 2, 0]))
    x = torch.ones((3, HID), dtype=torch.bfloat16, device=DEV)
    y = model.forward(x, hts.kv_step(cached, added, free, table, PAGE, 3), table)
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isfinite(y[0]).all())


def test_block_refuses_shapes_that_do_not_fit():
    model = Model(torch.bfloat16, seed=6)
    layer, st = model.layers[0], hts.KVStep.buffers(2, 2, DEV)
    table = torch.zeros((2, 4), dtype=torch.int32, device=DEV)
    x = torch.zeros((2, HID), dtype=torch.bfloat16, device=DEV)
    for change in (dict(k=layer.weights["q"]), dict(down=layer.weights["up"]), dict(o=layer.weights["k"]),
                   dict(v=hts.unpack(layer.weights["v"]).half())):
        with pytest.raises(hts.HTSError):
            block.Layer({**layer.weights, **change}, layer.cache, layer.input_norm, layer.mlp_norm)
    with pytest.raises(hts.HTSError):
        block.Layer({n: w for n, w in layer.weights.items() if n != "up"}, layer.cache, layer.input_norm, layer.mlp_norm)
    for bad in (x.half(), x[:1], x[:, :256]):
        with pytest.raises(hts.HTSError):
            block.decode(bad, None, layer, st, table, model.plan)


def test_block_refuses_before_it_writes_to_the_cache():
    # what only attention would refuse, behind the cache write of the same step
    model = Model(torch.bfloat16, seed=6)
    layer = model.layers[0]
    args = layer.cache, layer.input_norm, layer.mlp_norm
    q, o = (torch.zeros(s, dtype=torch.bfloat16, device=DEV) for s in ((3 * DIM, HID), (HID, 3 * DIM)))
    for change, kw in ((dict(q=q, o=o), {}), ({}, dict(window=-1)), ({}, dict(attn_scale=float("nan"))),
                       ({}, dict(attn_scale=float("inf")))):
        with pytest.raises(hts.HTSError):
            block.Layer({**layer.weights, **change}, *args, **kw)
    block.Layer({**layer.weights, "q": q[:2 * DIM], "o": o[:, :2 * DIM].contiguous()}, *args, window=5, attn_scale=0.1)
