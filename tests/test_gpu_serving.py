"""GPU parity of the steps around the products: page step, rotary positions with the cache write, paged
attention, residual norm -- each against its 64-bit form (serving_ref), with what must stay as it was
held in canary values.  Tolerances: half a rounding step of the output (finfo.eps / 2 relative) plus the
bound on the 32-bit arithmetic that the reference carries."""
import numpy as np
import pytest
import torch

import serving_ref as ref
import tile_gemm_amd as hts
from helpers import DEV, say

pytestmark = pytest.mark.gpu
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}


def f64(t):
    return t.float().double().cpu().numpy() if t.dtype != torch.float64 else t.cpu().numpy()


def normal(g, shape, dtype, sigma=1.0):
    return torch.from_numpy(g.standard_normal(shape).astype(np.float32) * np.float32(sigma)).to(DEV).to(TORCH[dtype])


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def strided(t, pad, fill=7.0):
    """The same matrix with a leading dimension pad entries longer, and the buffer it lies in."""
    big = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=DEV)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]], big


# ---- page step -------------------------------------------------------------

def _step_case(B, page, width, seed, mode):
    g = np.random.default_rng(seed)
    cap = width * page
    cached = g.integers(0, max(1, cap - page), B)
    added = g.integers(0, 3 * page, B) * (g.random(B) < 0.7)
    if mode == "decode":
        added = np.ones(B, np.int64)
    if mode == "wild":                       # negative counts, lengths past the row, past 32 bits when added up
        cached = np.where(g.random(B) < 0.3, g.integers(-50, 2 * cap, B), cached)
        cached = np.where(g.random(B) < 0.1, 2 ** 31 - 1, cached)
        added = np.where(g.random(B) < 0.2, -3, added)
    n_free = B * width if mode != "short" else max(1, B // 2)
    free = g.permutation(n_free + 5)[:n_free]
    if mode == "wild":
        free = np.where(g.random(n_free) < 0.1, -7, free)
    table = g.integers(-1, 1000, (B, width + 3))
    tokens = int(np.maximum(added, 0).sum()) + {"decode": 0, "mixed": 9, "short": 5, "wild": 40}[mode]
    if mode == "mixed" and B % 2:
        tokens = max(0, tokens // 2)         # a capacity below the batch's tokens
    return cached, added, free, table, tokens


@pytest.mark.parametrize("mode", ["decode", "mixed", "short", "wild"])
@pytest.mark.parametrize("B,page,width", [(1, 16, 1), (3, 16, 40), (64, 16, 7), (65, 64, 5), (257, 16, 9),
                                          (1000, 128, 3), (4096, 1024, 2)])
def test_kv_step(B, page, width, mode):
    cached, added, free, table, tokens = _step_case(B, page, width, B + page, mode)
    head = {"decode": 0, "mixed": 2, "short": 0, "wild": -4}[mode]
    say(f"[kv_step] B={B} page={page} width={width} {mode} tokens={tokens}")
    t = i32(table)
    st = hts.kv_step(i32(cached), i32(added), i32(free), t[:, :width], page, tokens,
                     free_head=None if mode == "decode" else i32([head]))
    want = ref.kv_step(cached.tolist(), added.tolist(), page, free.tolist(), head, table.tolist(), width, tokens)
    got = (t.cpu().tolist(), st.lengths.cpu().tolist(), st.starts.cpu().tolist(), st.slots.cpu().tolist(),
           st.positions.cpu().tolist(), int(st.head))
    for name, a, b in zip(("table", "lengths", "starts", "slots", "positions", "head"), got, want):
        assert a == b, name


def test_kv_step_of_no_requests_and_no_tokens():
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    st = hts.kv_step(e, e, e, torch.empty((0, 4), dtype=torch.int32, device=DEV), 16, 5, free_head=i32([3]))
    assert st.starts.tolist() == [0] and st.slots.tolist() == [-1] * 5 and st.positions.tolist() == [-1] * 5
    assert int(st.head) == 3
    t = i32([[5, -1, -1]])
    st = hts.kv_step(i32([16]), i32([17]), i32([8, 9]), t, 16, 0)
    assert t.tolist() == [[5, 8, 9]] and st.lengths.tolist() == [33] and st.starts.tolist() == [0, 17]


def test_kv_step_grows_a_running_batch():
    # steps one after another, each from the last one's lengths and head: every token keeps its slot
    B, page, width = 5, 16, 6
    free = torch.randperm(B * width, device=DEV).int()
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    cached, head = torch.zeros(B, dtype=torch.int32, device=DEV), i32([0])
    seen = {}
    for add in ([20, 1, 0, 33, 16], [1] * 5, [1] * 5, [0, 15, 40, 1, 1], [1] * 5):
        st = hts.kv_step(cached, i32(add), free, table, page, sum(add), free_head=head)
        b = np.repeat(np.arange(B), add)
        for who, pos, slot in zip(b, st.positions.tolist(), st.slots.tolist()):
            assert slot >= 0 and (int(who), pos) not in seen and slot not in seen.values()
            seen[(int(who), pos)] = slot
        cached, head = st.lengths, st.head
        rows = table.cpu().numpy()
        for (who, pos), slot in seen.items():
            assert rows[who, pos // page] * page + pos % page == slot
    assert cached.tolist() == [23, 19, 43, 37, 20]


# ---- rotary ----------------------------------------------------------------

ROPE = [  # dim, rot, layout, q heads, k heads, tokens
    (128, 128, "half", 32, 32, 1), (128, 128, "interleaved", 8, 2, 37), (64, 64, "half", 3, 1, 5),
    (80, 40, "half", 5, 5, 9), (96, 48, "interleaved", 4, 1, 3), (256, 64, "half", 2, 1, 300),
    (256, 256, "interleaved", 2, 2, 4), (8, 8, "half", 1, 1, 2), (192, 16, "half", 3, 2, 17),
    (88, 24, "interleaved", 7, 3, 65), (128, 8, "half", 40, 8, 2),
]


def _positions(g, T):
    p = g.integers(0, 100000, T)
    far = [0, 1, 2 ** 31 - 1, 1000003, 131071]
    p[:min(T, 5)] = far[:min(T, 5)]
    return p


# The angle in turns is below 2^29; the plan's and the product's roundings leave at most 2^-23 of a turn
# there, the reduced turn's own rounding and the sine's 2^-24 each: under 2^-20 in radians with the factor
# 2 pi, and four more roundings of 2^-24 in the rotation.
TURN = 2.0 ** -19


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,rot,layout,hq,hk,T", ROPE)
def test_rope(dtype, dim, rot, layout, hq, hk, T):
    g = np.random.default_rng(dim + rot + T)
    q, k = normal(g, (T, hq * dim), dtype), normal(g, (T, hk * dim), dtype)
    pos = _positions(g, T)
    if T > 8:
        pos[T // 2] = -1                       # a skipped row
    say(f"[rope] {dtype} dim={dim} rot={rot} {layout} {hq}/{hk} T={T}")
    plan = hts.rope_plan(dim, rot, theta=500000.0, layout=layout, rule="linear", factor=1.5, magnitude=1.25, device=DEV)
    turns = ref.rope_turns(rot, 500000.0, "linear", 1.5)
    qs, ks = strided(q, 24)[0], strided(k, 8)[0]
    qo, qbig = strided(torch.full_like(q, 3.0), 16)
    ko, kbig = strided(torch.full_like(k, 3.0), 40)
    hts.rope(qs, ks, i32(pos), plan, q_out=qo, k_out=ko)
    for x, got, big in ((q, qo, qbig), (k, ko, kbig)):
        want, size = ref.rope(f64(x), pos, turns, dim, layout, 1.25)
        live = pos >= 0
        err = np.abs(f64(got) - want)
        tol = ref.EPS[dtype] / 2 * np.abs(want) + TURN * size + ref.TINY[dtype]
        assert np.all(err[live] <= tol[live]), float((err - tol)[live].max())
        assert np.all(f64(got)[~live] == 3.0)
        assert torch.all(big[:, x.shape[1]:] == 7.0)
    # in place, q alone and k alone: the same bits
    q2, k2 = q.clone(), k.clone()
    hts.rope(q2, None, i32(pos), plan)
    hts.rope(None, k2, i32(pos), plan)
    live = torch.from_numpy(pos >= 0).to(DEV)
    assert torch.equal(q2[live], qo[live]) and torch.equal(k2[live], ko[live])
    assert torch.equal(q2[~live], q[~live])


@pytest.mark.parametrize("cache_dtype", ["same", "fp8"])
@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("dim,rot,layout,hq,hk,T", ROPE)
def test_rope_cache(dim, rot, layout, hq, hk, T, order, cache_dtype):
    dtype = "bf16" if T % 2 else "f16"
    g = np.random.default_rng(dim * 3 + rot + T)
    page = 16 if T % 3 else 32
    pages = -(-T // page) + 2
    qkv = normal(g, (T, (hq + 2 * hk) * dim), dtype, 3.0)
    q, k, v = qkv[:, :hq * dim], qkv[:, hq * dim:(hq + hk) * dim], qkv[:, (hq + hk) * dim:]
    pos = _positions(g, T)
    slots = g.permutation(pages * page)[:T]
    if T > 8:
        pos[3], slots[4], slots[5], slots[6] = -1, -1, pages * page, 2 ** 40
    ct = dtype if cache_dtype == "same" else "fp8"
    ks = vs = None
    if ct == "fp8":
        ks = torch.from_numpy(g.uniform(0.01, 2.0, hk).astype(np.float32)).to(DEV)
        vs = torch.from_numpy(g.uniform(0.01, 2.0, hk).astype(np.float32)).to(DEV)
    cache = hts.kv_cache(pages, page, hk, dim, TORCH[ct], DEV, order, ks, vs)
    for c in (cache.k, cache.v):
        c.view(torch.uint8).fill_(0x11)
    before = [c.view(torch.uint8).clone() for c in (cache.k, cache.v)]
    say(f"[rope_cache] {dtype} cache={ct} {order} dim={dim} rot={rot} {layout} {hq}/{hk} T={T}")
    plan = hts.rope_plan(dim, rot, layout=layout, device=DEV)
    qo = torch.full((T, hq * dim), 3.0, dtype=TORCH[dtype], device=DEV)
    hts.rope_cache(q, k, v, i32(pos), torch.from_numpy(slots).to(DEV), plan, cache, q_out=qo)
    turns = ref.rope_turns(rot)
    live = pos >= 0
    want, size = ref.rope(f64(q), pos, turns, dim, layout, 1.0)
    tol = ref.EPS[dtype] / 2 * np.abs(want) + TURN * size + ref.TINY[dtype]
    assert np.all((np.abs(f64(qo) - want) <= tol)[live]) and np.all(f64(qo)[~live] == 3.0)
    put = live & (slots >= 0) & (slots < pages * page)
    where = (slots[put] // page, slots[put] % page)
    want, size = ref.rope(f64(k), pos, turns, dim, layout, 1.0)
    for c, x, sz, s in ((cache.k, want, size, ks), (cache.v, f64(v), np.zeros_like(size), vs)):
        got = f64(c)[where]
        x, sz = x.reshape(T, hk, dim)[put], sz.reshape(T, hk, dim)[put]
        if ct == "fp8":
            sc = np.ones(hk) if s is None else f64(s)
            x, sz = x / sc[:, None], sz / sc[:, None]
            x = np.clip(x, -448.0, 448.0)
            # half a step of e4m3 (2^-4 of the value, 2^-10 among its subnormals) and the division's rounding
            tol = 2.0 ** -4 * np.abs(x) + 2.0 ** -10 + TURN * sz + 2.0 ** -23 * np.abs(x)
        else:
            tol = ref.EPS[dtype] / 2 * np.abs(x) + TURN * sz + ref.TINY[dtype]
        assert np.all(np.abs(got - x) <= tol)
    # nothing but those slots was written
    for c, b in zip((cache.k, cache.v), before):
        now = c.view(torch.uint8).clone()
        now[torch.from_numpy(where[0]).to(DEV), torch.from_numpy(where[1]).to(DEV)] = 0x11
        assert torch.equal(now, b)


def test_e4m3_cache_rounds_to_nearest_even_and_saturates():
    # v is stored unturned: every 16-bit value in order of the format, against torch's own E4M3 conversion
    bits = torch.arange(65536, dtype=torch.int32, device=DEV).to(torch.int16)
    for dt in (torch.bfloat16, torch.float16):
        v = bits.view(dt).view(256, 256)
        k = torch.zeros_like(v)
        cache = hts.kv_cache(16, 16, 1, 256, torch.float8_e4m3fn, DEV)
        plan = hts.rope_plan(256, 8, device=DEV)
        hts.rope_cache(k.clone(), k, v, torch.zeros(256, dtype=torch.int32, device=DEV),
                       torch.arange(256, device=DEV), plan, cache)
        got = cache.v.reshape(256, 256).float()
        f = v.float()
        want = f.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
        assert torch.equal(torch.isnan(got), torch.isnan(f))
        ok = ~torch.isnan(f)
        assert torch.equal(got[ok], want[ok])


@pytest.mark.parametrize("cache_dtype", ["bf16", "fp8"])
def test_rope_cache_of_a_row_per_request(cache_dtype):
    # requests that add no token, one, two, one past the capacity: rows of the second kind as if token by token
    dim, hq, hk, page = 64, 4, 2, 16
    g = np.random.default_rng(9)
    starts = [0, 1, 1, 2, 3, 5, 6, 6, 7, 8]               # requests 1 and 6 add none, 4 two, the last's token is past 7
    live, none, lost = [0, 2, 3, 5, 7], [1, 6], [4, 8]
    B, tokens = len(starts) - 1, 7
    q, k, v = (normal(g, (B, h * dim), "bf16") for h in (hq, hk, hk))
    pos, slots = i32([5, 9, -1, 100, 101, 77, 3]), torch.tensor([40, 3, 17, 18, 19, 60, -1], device=DEV)
    plan = hts.rope_plan(dim, 32, device=DEV)
    caches = [hts.kv_cache(4, page, hk, dim, TORCH[cache_dtype], DEV) for _ in range(2)]
    out = torch.full_like(q, 3.0)
    hts.rope_cache(q, k, v, pos, slots, plan, caches[0], q_out=out, starts=i32(starts))
    at = torch.tensor([starts[b] for b in live], device=DEV)
    want = torch.full_like(q, 3.0)
    rows = torch.tensor(live, device=DEV)
    part = torch.full((len(live), hq * dim), 3.0, dtype=q.dtype, device=DEV)
    hts.rope_cache(q[rows], k[rows], v[rows], pos[at], slots[at], plan, caches[1], q_out=part)
    want[rows] = part
    assert torch.equal(out[rows], want[rows]) and torch.all(out[none] == 3.0) and torch.all(out[3] == 3.0)
    for a, b in zip((caches[0].k, caches[0].v), (caches[1].k, caches[1].v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and bool((a.float() != 0).any())
    assert bool(torch.isnan(out[lost].view(2, hq, dim)[..., :32]).all())
    for bad in (i32(starts[:-1]), i32([]), i32(starts).long()):
        with pytest.raises(hts.HTSError):
            hts.rope_cache(q, k, v, pos, slots, plan, caches[0], q_out=out, starts=bad)


def test_rope_of_more_tokens_than_a_grid_axis_takes():
    # past 2^24 workgroups of 256 threads: the rows of a small call, over and over
    P, n = 4096, 4099
    g = np.random.default_rng(8)
    q, k, v = (normal(g, (P, 8), "bf16") for _ in range(3))
    pos = i32(g.integers(-1, 100000, P))
    plan = hts.rope_plan(8, device=DEV)
    want_q, want_k = hts.rope(q.clone(), k.clone(), pos, plan)
    T = n * P
    qq, kk, pp = q.repeat(n, 1), k.repeat(n, 1), pos.repeat(n)
    hts.rope(qq, kk, pp, plan)
    assert torch.equal(qq.view(n, P, 8), want_q.expand(n, P, 8)) and torch.equal(kk.view(n, P, 8), want_k.expand(n, P, 8))
    # and into a cache of as many tokens, where a skipped token leaves its place as it was
    cache = hts.kv_cache(T // 1024, 1024, 1, 8, torch.bfloat16, DEV)
    qq = q.repeat(n, 1)
    hts.rope_cache(qq, k.repeat(n, 1), v.repeat(n, 1), pp, torch.arange(T, device=DEV), plan, cache)
    live = (pos >= 0)[:, None]
    zero = torch.zeros_like(k)
    assert torch.equal(qq.view(n, P, 8), want_q.expand(n, P, 8))
    assert torch.equal(cache.k.view(n, P, 8), torch.where(live, want_k, zero).expand(n, P, 8))
    assert torch.equal(cache.v.view(n, P, 8), torch.where(live, v, zero).expand(n, P, 8))


# ---- attention -------------------------------------------------------------

ATTN = [  # dim, q heads, k heads, page, order, cache, window, lengths
    (128, 32, 32, 16, "token", "same", 0, [1]),
    (128, 32, 8, 16, "token", "same", 0, [0, 1, 15, 16, 17, 31, 32, 33, 100, 257]),
    (128, 8, 8, 64, "head", "same", 0, [63, 64, 65, 0, 500]),
    (128, 40, 8, 32, "head", "fp8", 0, [7, 0, 300, 1111]),
    (64, 14, 2, 16, "token", "same", 0, [5, 129, 640]),
    (64, 6, 3, 128, "head", "fp8", 0, [1, 128, 129, 1000]),
    (80, 5, 5, 16, "token", "same", 0, [33, 1, 90]),
    (96, 12, 4, 16, "head", "fp8", 0, [48, 700]),
    (192, 8, 1, 256, "token", "same", 0, [2, 255, 256, 257]),
    (256, 16, 1, 16, "token", "same", 0, [0, 400, 3]),
    (256, 6, 2, 1024, "head", "fp8", 0, [1500, 1]),
    (8, 4, 4, 16, "token", "same", 0, [40, 2]),
    (8, 9, 3, 16, "head", "fp8", 0, [40, 2]),
    (128, 40, 2, 16, "token", "same", 0, [700, 50, 0]),      # more than 16 query heads to a cache head
    (104, 33, 1, 32, "head", "same", 0, [513, 64]),
    (128, 8, 2, 16, "token", "same", 1, [50, 0, 1, 3000]),   # windows
    (128, 8, 2, 32, "head", "fp8", 100, [99, 100, 101, 2500]),
    (64, 4, 4, 16, "token", "same", 1000, [5000, 999, 17]),
    (128, 8, 1, 16, "token", "same", 0, [20000, 3, 0, 9000]),  # lengths that are split
    (128, 16, 2, 64, "token", "fp8", 0, [12345]),
    (72, 3, 3, 16, "head", "same", 5000, [16384, 40]),
]


def _attn_case(dim, hq, hk, page, order, cache, lengths, dtype, seed, spare=2):
    g = np.random.default_rng(seed)
    B, width = len(lengths), -(-max(max(lengths), 1) // page) + 1
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + spare
    ct = dtype if cache == "same" else "fp8"
    ks = vs = None
    if ct == "fp8":
        ks = torch.from_numpy(g.uniform(0.2, 2.0, hk).astype(np.float32)).to(DEV)
        vs = torch.from_numpy(g.uniform(0.2, 2.0, hk).astype(np.float32)).to(DEV)
    c = hts.kv_cache(pages, page, hk, dim, TORCH[ct], DEV, order, ks, vs)
    # every place holds NaN but those of the requests' tokens
    c.k.view(torch.uint8).fill_(0x7F if ct == "fp8" else 0xFF)
    c.v.view(torch.uint8).fill_(0x7F if ct == "fp8" else 0xFF)
    ids = g.permutation(pages)
    table = np.full((B, width + 2), -1)
    at = 0
    gg = torch.Generator(device=DEV)
    gg.manual_seed(seed)
    for b, n in enumerate(lengths):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
        if n:
            t = torch.arange(n, device=DEV)
            rows = torch.from_numpy(table[b]).to(DEV)[t // page]
            for x in (c.k, c.v):
                val = torch.randn((n, hk, dim), generator=gg, device=DEV).to(TORCH[ct])
                if ct == "fp8":
                    x.view(torch.uint8)[rows, t % page] = val.view(torch.uint8)
                else:
                    x[rows, t % page] = val
    q = normal(g, (B, hq * dim), dtype)
    return q, c, table, width


def _check_attn(q, c, table, width, lengths, hq, window, scale, out, lse, dtype):
    k, v = f64(c.k), f64(c.v)
    if c.k_scale is not None:
        k, v = k * f64(c.k_scale)[:, None], v * f64(c.v_scale)[:, None]
    B = len(lengths)
    want, wl, err, el = ref.attn(f64(q).reshape(B, hq, c.dim), k, v, table[:, :width], lengths, c.page, scale, window,
                                 c.heads)
    got = f64(out).reshape(B, hq, c.dim)
    tol = ref.EPS[dtype] / 2 * np.abs(want) + err + ref.TINY[dtype]
    bad = np.abs(got - want) - tol
    assert np.all(bad <= 0), f"out off by {float(np.nanmax(bad)):.3e} past its tolerance (NaN: {np.isnan(got).sum()})"
    if lse is not None:
        g = f64(lse)
        empty = np.isinf(wl)
        assert np.array_equal(g[empty], wl[empty])
        assert np.all(np.abs(g - wl)[~empty] <= el[~empty]), float((np.abs(g - wl) - el)[~empty].max())
    return want


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,hq,hk,page,order,cache,window,lengths", ATTN)
def test_paged_attn(dim, hq, hk, page, order, cache, window, lengths, dtype):
    q, c, table, width = _attn_case(dim, hq, hk, page, order, cache, lengths, dtype, dim + hq + page)
    say(f"[attn] {dtype} dim={dim} {hq}/{hk} page={page} {order} {cache} window={window} lengths={lengths}")
    B = len(lengths)
    qs = strided(q, 16)[0]
    out, big = strided(torch.full_like(q, 5.0), 8)
    lse = torch.empty((B, hq), dtype=torch.float32, device=DEV)
    t = i32(table)[:, :width]
    scale = 0.7 * dim ** -0.5
    hts.paged_attn(qs, c, t, i32(lengths), scale=scale, window=window, out=out, lse=lse)
    _check_attn(q, c, table, width, lengths, hq, window, scale, out, lse, dtype)
    assert torch.all(big[:, q.shape[1]:] == 7.0)
    # the same call again: the same bits; in place, and unsplit for lack of a workspace: within the tolerance
    again = hts.paged_attn(q, c, t, i32(lengths), scale=scale, window=window)
    assert torch.equal(again, out)
    q2 = q.clone()
    hts.paged_attn(q2, c, t, i32(lengths), scale=scale, window=window, out=q2)
    assert torch.equal(q2, out)
    q2 = q.clone()
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    hts.paged_attn(q2, c, t, i32(lengths), scale=scale, window=window, out=q2, workspace=small)
    _check_attn(q, c, table, width, lengths, hq, window, scale, q2, None, dtype)


def test_paged_attn_of_one_cache_head_in_either_order():
    # the same memory in "token" and in "head" order (they differ in a stride that one head does not use): the same bits
    lengths = [9000, 70, 0, 5000]
    q, c, table, width = _attn_case(128, 8, 1, 16, "token", "same", lengths, "bf16", 21)
    other = hts.KVCache(*(x.as_strided(x.shape, (x.stride(0), x.stride(1), 16 * 128, 1)) for x in (c.k, c.v)))
    args = i32(table)[:, :width], i32(lengths)
    assert torch.equal(hts.paged_attn(q, c, *args), hts.paged_attn(q, other, *args))


def test_paged_attn_leaves_out_what_no_page_holds():
    # entries of -1, ids past the cache and lengths past the table (and negative) within the requests
    lengths = [200, 90, 33, 64]
    q, c, table, width = _attn_case(128, 8, 2, 16, "token", "same", lengths, "bf16", 5)
    table[0, 3], table[0, 4], table[1, 0:6], table[2, 0] = -1, 10 ** 6, -5, 2 ** 31 - 1
    given = [200, 90, 33, -64]
    lse = torch.empty((4, 8), dtype=torch.float32, device=DEV)
    out = hts.paged_attn(q, c, i32(table)[:, :width], i32(given), scale=0.1, lse=lse)
    want = _check_attn(q, c, table, width, given, 8, 0, 0.1, out, lse, "bf16")
    assert np.all(want[1] == 0) and np.all(want[3] == 0) and np.any(want[2] != 0)
    # a length past what the table's width holds ends there
    cut = -(-64 // 16)
    out = hts.paged_attn(q[3:], c, i32(table)[3:, :cut], i32([10 ** 9]), scale=0.1)
    _check_attn(q[3:], c, table[3:], cut, [64], 8, 0, 0.1, out, None, "bf16")


def test_paged_attn_far_offsets():
    # an 8-bit cache of 5 GB: offsets past 2^32 elements
    page, hk, dim = 64, 8, 128
    pages = (5 << 30) // (page * hk * dim)
    k = torch.empty((pages, page, hk, dim), dtype=torch.float8_e4m3fn, device=DEV)
    v = torch.empty_like(k)
    g = np.random.default_rng(1)
    use = [pages - 1, 0, pages - 2, pages // 2, 70000]
    small = hts.kv_cache(5, page, hk, dim, torch.float8_e4m3fn, DEV)
    for big, sm in ((k, small.k), (v, small.v)):
        sm.copy_(normal(g, sm.shape, "f32").to(torch.float8_e4m3fn))
        for i, p in enumerate(use):
            big.view(torch.uint8)[p] = sm.view(torch.uint8)[i]
    q = normal(g, (1, 16 * dim), "bf16")
    n = i32([5 * page - 3])
    a = hts.paged_attn(q, hts.KVCache(k, v), i32([use]), n)
    b = hts.paged_attn(q, small, i32([[0, 1, 2, 3, 4]]), n)
    assert torch.equal(a, b) and bool((a != 0).any())
    # and the cache write of the rotary step there
    plan = hts.rope_plan(dim, device=DEV)
    x = normal(g, (2, hk * dim), "bf16")
    slots = torch.tensor([(pages - 1) * page + 5, 3 * page], device=DEV)
    hts.rope_cache(x.clone(), x, x, i32([9, 10]), slots, plan, hts.KVCache(k, v))
    hts.rope_cache(x.clone(), x, x, i32([9, 10]), torch.tensor([5, 64], device=DEV), plan, small)
    assert torch.equal(k.view(torch.uint8)[pages - 1, 5], small.k.view(torch.uint8)[0, 5])
    assert torch.equal(v.view(torch.uint8)[3, 0], small.v.view(torch.uint8)[1, 0])


def test_paged_attn_extreme_scores():
    # scores in the tens of thousands, all equal scores, and rows whose scores are all minus infinity
    page, dim = 16, 128
    c = hts.kv_cache(3, page, 1, dim, torch.float16, DEV)
    g = np.random.default_rng(2)
    c.k.copy_(normal(g, c.k.shape, "f16", 100.0))
    c.v.copy_(normal(g, c.v.shape, "f16"))
    table = np.array([[2, 0, 1]])
    q = normal(g, (1, 4 * dim), "f16", 30.0)
    q[0, dim:2 * dim] = 0
    out = hts.paged_attn(q, c, i32(table), i32([40]), scale=1.0)
    k, v = f64(c.k), f64(c.v)
    want, _, err, _ = ref.attn(f64(q).reshape(1, 4, dim), k, v, table, [40], page, 1.0, 0, 1)
    tol = ref.EPS["f16"] / 2 * np.abs(want) + err + ref.TINY["f16"]
    assert np.all(np.abs(f64(out).reshape(1, 4, dim) - want) <= tol)
    c.k[2, 5, 0, 0] = float("inf")            # q.k = -inf for that token alone: it gets no weight
    q = torch.zeros((1, dim), dtype=torch.float16, device=DEV)
    q[0, 0] = -1.0
    lse = torch.empty((1, 1), device=DEV)
    out = hts.paged_attn(q, c, i32(table), i32([40]), scale=1.0, lse=lse)
    kk = k.copy()
    kk[2, 5] = 0
    t = np.array([i for i in range(40) if i != 5])
    ids = table[0, t // page]
    s = -kk[ids, t % page, 0, 0]
    p = np.exp(s - s.max())
    want = p @ v[ids, t % page, 0] / p.sum()
    assert np.all(np.abs(f64(out)[0] - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -14 * np.abs(v).max())
    c.k[..., 0] = float("inf")                # every score minus infinity: no weight at all
    out = hts.paged_attn(q, c, i32(table), i32([40]), scale=1.0, lse=lse)
    assert torch.all(out == 0) and float(lse) == -np.inf
    c.k.zero_()
    c.v[2, 7, 0, 3] = float("nan")            # NaN in a token that counts does show
    out = hts.paged_attn(q, c, i32(table), i32([40]), scale=1.0)
    assert bool(torch.isnan(out[0, 3])) and int(torch.isnan(out).sum()) == 1


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_paged_attn_small_weights_add_up(dtype):
    # one token of weight 1 and value 0, and 100000 of weight e^-18 (2^-26) and value 1: together 1.5e-3
    page, n = 64, 100001
    pages = -(-n // page)
    c = hts.kv_cache(pages, page, 1, 64, TORCH[dtype], DEV)
    c.k[..., 0] = -18.0
    c.v.fill_(1.0)
    for first in (0, 70000):                    # the large weight first, and late (in another run)
        c.k[first // page, first % page, 0, 0] = 0.0
        c.v[first // page, first % page] = 0.0
        q = torch.zeros((1, 2 * 64), dtype=TORCH[dtype], device=DEV)
        q[0, 0] = 1.0
        q[0, 64] = 0.5                           # the second head: weights e^-9
        lse = torch.empty((1, 2), device=DEV)
        out = hts.paged_attn(q, c, torch.arange(pages, dtype=torch.int32, device=DEV)[None], i32([n]), scale=1.0, lse=lse)
        got = f64(out)[0].reshape(2, 64)
        for h, w in enumerate((np.exp(-18.0), np.exp(-9.0))):
            want = (n - 1) * w / (1 + (n - 1) * w)
            # half a step of the type, the weights' 2^-16, and 100000 additions in 32 bits over 96 lanes and more
            tol = (ref.EPS[dtype] / 2 + 2.0 ** -16 + n / 96 * 2.0 ** -24) * want
            assert np.all(np.abs(got[h] - want) <= tol), (first, h, got[h][:2], want)
            assert abs(float(lse[0, h]) - np.log(1 + (n - 1) * w)) <= 1e-4
        c.k[first // page, first % page, 0, 0] = -18.0
        c.v[first // page, first % page] = 1.0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_paged_attn_small_weights_beside_a_large_one(dtype, dim):
    # one wave forms large and small weights together: the call is not split (no room for its parts), and every wave
    # starts with a token of weight 1 and value 0; 100000 others have weights e^-9 to e^-20.25 and the value 100
    page, n, heavy, v = 64, 100008, 8, 100.0
    pages = -(-n // page)
    c = hts.kv_cache(pages, page, 1, dim, TORCH[dtype], DEV)
    c.k[..., 0] = -18.0
    c.v.fill_(v)
    c.k[0, 0:16 * heavy:16, 0, 0] = 0.0          # waves start at tokens 0, 16, 32, 48 or 0, 32, 64, 96
    c.k[1, 0:16 * heavy - 64:16, 0, 0] = 0.0
    c.v[0, 0:64:16] = 0.0
    c.v[1, 0:64:16] = 0.0
    by = [0.5, 1.0, 1.0625, 1.125]               # scores of -9, -18, -19.125, -20.25: exact in either type
    q = torch.zeros((1, len(by) * dim), dtype=TORCH[dtype], device=DEV)
    for h, x in enumerate(by):
        q[0, h * dim] = x
    lse = torch.empty((1, len(by)), device=DEV)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    out = hts.paged_attn(q, c, table, i32([n]), scale=1.0, lse=lse, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    got = f64(out)[0].reshape(len(by), dim)
    for h, x in enumerate(by):
        w = np.exp(-18.0 * x)
        small = (n - heavy) * w
        want = small * v / (heavy + small)
        # half a step of the type; a weight's own 2^-21, or 2^-43 of the largest weight; the exponential's argument
        # (|s| log2 e below 32: 2^-20 of its rounding) and its last place; sums of a lane's pairs (16 lanes share the
        # tokens) and of a wave's steps of 16 tokens, in 32 bits
        tol = ref.EPS[dtype] / 2 + 2.0 ** -21 + 2.0 ** -43 / w + 2.0 ** -19 + (n / 32 + n / 64) * 2.0 ** -24
        assert np.all(np.abs(got[h] - want) <= tol * want), (dim, x, got[h][:2], want, tol)
        assert abs(float(lse[0, h]) - np.log(heavy + small)) <= 2.0 ** -18 + n / 32 * 2.0 ** -24


@pytest.mark.parametrize("cache", ["same", "fp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 192])
def test_paged_attn_values_that_cancel(dtype, dim, cache):
    # two tokens whose weighted values nearly cancel: what is left shows the weights' own precision.  A head's weights
    # are 1 and about a / b, its values -a and b.
    page = 16
    ratio = [(8, 15, -1), (8, 15, -3), (8, 13, 1), (8, 15, 1), (9, 14, 3), (9, 11, -3), (11, 13, -1), (9, 13, 3)]
    hk = len(ratio)
    ct = TORCH[dtype] if cache == "same" else TORCH["fp8"]
    k, v = torch.zeros((1, page, hk, dim)), torch.zeros((1, page, hk, dim))
    for h, (a, b, off) in enumerate(ratio):
        left = np.log(a / b * (1 + off * 2.0 ** -13))   # the second token's score, in as many entries as it takes
        for d in range(8):
            part = torch.tensor(left, dtype=torch.float32).to(ct).float()
            k[0, 1, h, d] = part
            left -= float(part)
        v[0, 0, h], v[0, 1, h] = -a, b
    c = hts.KVCache(k.to(ct).to(DEV), v.to(ct).to(DEV))
    q = torch.ones((1, hk * dim), dtype=TORCH[dtype], device=DEV)
    got = f64(hts.paged_attn(q, c, i32([[0]]), i32([2]), scale=1.0))[0].reshape(hk, dim)
    kk, vv = f64(c.k)[0], f64(c.v)[0]
    for h in range(hk):
        p = np.exp(np.array([0.0, kk[1, h].sum()]))
        want = p @ vv[:2, h] / p.sum()
        # half a step of the type, and relative to the second value's weight: the weight's 2^-21; its argument, up to
        # 8 (2^-22 ln 2); the exponential's last place (2^-23); a score below 1 summed from 8 terms that shrink by 2^-4
        # and more, and scaled (2^-23); two sums (2^-23 together)
        tol = ref.EPS[dtype] / 2 * np.abs(want) + (2.0 ** -21 + 0.7 * 2.0 ** -22 + 3 * 2.0 ** -23) * p[1] * vv[1, h] / p.sum()
        assert np.all(np.abs(got[h] - want) <= tol), (h, got[h][:2], want[:2], tol[:2])


@pytest.mark.parametrize("lengths", [[100, 3], [9000, 70, 0]])
def test_paged_attn_in_a_graph(lengths):
    # captured once at one set of lengths, replayed at others with eager work in between
    q, c, table, width = _attn_case(128, 16, 2, 16, "token", "same", lengths, "bf16", 11)
    t, n = i32(table)[:, :width].contiguous(), i32(lengths)
    eager = {}
    variants = [lengths, [x // 2 for x in lengths], [0] * len(lengths), [max(1, x - 1) for x in lengths]]
    for i, ls in enumerate(variants):
        eager[i] = hts.paged_attn(q, c, t, i32(ls)).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        hts.paged_attn(q, c, t, n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = hts.paged_attn(q, c, t, n)
    for rep in range(2):
        for i, ls in enumerate(variants):
            n.copy_(i32(ls))
            out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager[i]), f"replay {rep} at lengths {ls}"
            assert torch.equal(hts.paged_attn(q, c, t, i32(ls)), eager[i])


def test_steps_on_another_stream():
    lengths = [9000, 70, 0]
    q, c, table, width = _attn_case(128, 16, 2, 16, "token", "same", lengths, "bf16", 12)
    t, n = i32(table)[:, :width], i32(lengths)
    want = hts.paged_attn(q, c, t, n)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [hts.paged_attn(q, c, t, n, stream=s), hts.paged_attn(q, c, t, n, stream=s.cuda_stream)]
    x = normal(np.random.default_rng(0), (5, 64), "bf16")
    torch.cuda.synchronize()
    r, y = hts.residual_norm(x, x, pre=hts.Norm("rms"), stream=s)
    s.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], want)
    r2, y2 = hts.residual_norm(x, x, pre=hts.Norm("rms"))
    assert torch.equal(r, r2) and torch.equal(y, y2)


def test_paged_attn_joins_more_heads_than_a_grid_axis_takes():
    # 4096 requests of 4352 heads: the join takes 2.2 million workgroups; the one request that is cut lies past 2^21
    B, hk, hq, dim, page, long = 4096, 128, 4352, 128, 16, 4090
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    c = hts.KVCache(*(torch.randn((8, page, hk, dim), generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2)))
    n = torch.ones(B, dtype=torch.int32, device=DEV)
    n[long] = 134400
    width = 134400 // page
    table = torch.randint(0, 8, (B, width), generator=g, device=DEV, dtype=torch.int32)
    q = torch.randn((B, hq * dim), generator=g, device=DEV, dtype=torch.bfloat16)
    assert c.workspace_bytes(B, hq, width) > 0
    out = hts.paged_attn(q, c, table, n)
    rest = torch.arange(B, device=DEV) != long
    # a request of one token: its value, in every head of the group
    v = c.v[table[:, 0].long(), 0]
    for b in range(0, B, 512):
        want = v[b:b + 512, :, None].expand(-1, hk, hq // hk, dim).reshape(512, -1)
        assert torch.equal(out[b:b + 512][rest[b:b + 512]], want[rest[b:b + 512]])
    # the long one: the same call by itself, cut at other places (32-bit sums in another order, one rounding each)
    alone = hts.paged_attn(q[long:long + 1], c, table[long:long + 1], n[long:long + 1])
    assert torch.all((out[long] - alone[0]).abs().float() <= 2.0 ** -7 * alone[0].abs().float() + 2.0 ** -10)
    assert bool((out[long] != 0).any())


# ---- norm ------------------------------------------------------------------

NORM = [  # post, pre, gate, act, scale, residual
    ("none", "rms", "none", "none", 1.0, "same"), ("rms", "rms", "channel", "none", 0.5, "f32"),
    ("layer", "layer", "token", "sigmoid", 1.0, "same"), ("rms", "none", "token", "silu", -1.5, "f32"),
    ("none", "layer", "channel", "silu", 0.25, "same"), ("layer", "rms", "none", "none", 3.0, "f32"),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N", [(1, 8), (3, 64), (130, 128), (5, 520), (9, 1000), (2, 2048), (7, 2056), (300, 4096),
                                 (3, 4104), (4, 5120), (2, 8192), (3, 8200), (2, 16384), (2, 32768)])
@pytest.mark.parametrize("post,pre,gate,act,scale,res", NORM)
def test_residual_norm(M, N, post, pre, gate, act, scale, res, dtype):
    g = np.random.default_rng(M + N)
    rt = dtype if res == "same" else "f32"
    x, r = normal(g, (M, N), dtype, 2.0), normal(g, (M, N), rt, 3.0) + 0.5
    x[0] = 0                                   # a row of zeros
    if M > 2:
        r[1], x[1] = 5.0, 1.0                  # rows of one value
    gt = None if gate == "none" else normal(g, (N,) if gate == "channel" else (M, N), dtype)
    ws = {}
    for side, kind in (("post", post), ("pre", pre)):
        w = normal(g, (N,), dtype) if kind != "none" and N != 64 else None
        b = normal(g, (N,), dtype) if kind == "layer" else None
        ws[side] = (kind, 1e-5, w, b)
    say(f"[norm] {dtype} M={M} N={N} {post}/{pre} gate={gate}/{act} residual={rt}")
    norms = {s: hts.Norm(k, w, b, e) for s, (k, e, w, b) in ws.items()}
    xs, rs = strided(x, 8)[0], strided(r, 16)[0]
    ro, robig = strided(torch.zeros_like(r), 24)
    yo, yobig = strided(torch.zeros_like(x), 8)
    got_r, got_y = hts.residual_norm(xs, rs, norms["post"], norms["pre"], gt, act, scale, residual_out=ro, out=yo)
    arr = {s: (k, e, None if w is None else f64(w), None if b is None else f64(b)) for s, (k, e, w, b) in ws.items()}
    wr, er, wy, ey = ref.residual_norm(f64(x), f64(r), arr["post"], arr["pre"], None if gt is None else f64(gt), act, scale)
    assert np.all(np.abs(f64(got_r) - wr) <= ref.EPS[rt] / 2 * np.abs(wr) + er + ref.TINY[rt])
    assert np.all(np.abs(f64(got_y) - wy) <= ref.EPS[dtype] / 2 * np.abs(wy) + ey + ref.TINY[dtype])
    assert torch.all(robig[:, N:] == 7.0) and torch.all(yobig[:, N:] == 7.0)
    # in place over the residual and the block's output: the same bits
    r2, x2 = r.clone(), x.clone()
    hts.residual_norm(x2, r2, norms["post"], norms["pre"], gt, act, scale, residual_out=r2, out=x2)
    assert torch.equal(r2, got_r) and torch.equal(x2, got_y)


@pytest.mark.parametrize("N,n", [(8, 65537), (264, 513)])
def test_residual_norm_of_more_rows_than_a_grid_axis_takes(N, n):
    # 2^28 rows of 16 lanes and more are 2^32 threads; 2^21 rows of a workgroup each are an axis
    P = 4096
    g = np.random.default_rng(N)
    x, w = normal(g, (P, N), "bf16"), hts.Norm("layer", normal(g, (N,), "bf16"))
    want = hts.residual_norm(x, None, pre=w, keep_residual=False)[1]
    big = x.repeat(n, 1)
    assert big.shape[0] > (2 ** 28 if N == 8 else 2 ** 21)
    hts.residual_norm(big, None, pre=w, keep_residual=False, out=big)
    for i in range(0, n, 4096):
        part = big[i * P:(i + 4096) * P].view(-1, P, N)
        assert torch.equal(part, want.expand_as(part))


def test_residual_norm_parts():
    g = np.random.default_rng(3)
    x, r = normal(g, (6, 512), "bf16"), normal(g, (6, 512), "f32")
    n = hts.Norm("rms", normal(g, (512,), "bf16"), eps=1e-6)
    # no block: the plain norm of the residual; nothing kept
    keep, y = hts.residual_norm(None, r, pre=n, keep_residual=False, out_dtype=torch.bfloat16)
    assert keep is None and y.dtype == torch.bfloat16
    _, want = hts.residual_norm(torch.zeros_like(x), r, pre=n)
    assert torch.equal(y, want)
    # no residual: scale * block; no pre norm: no y
    keep, y = hts.residual_norm(x, None, scale=2.0)
    assert y is None and torch.equal(keep, x * 2)
    # the gate of one row through a view of stride 0, and through a vector
    gate = normal(g, (512,), "bf16")
    a, _ = hts.residual_norm(x, r, gate=gate)
    b, _ = hts.residual_norm(x, r, gate=gate.expand(6, 512))
    assert torch.equal(a, b)
    # y in place of the gate
    full = normal(g, (6, 512), "bf16")
    _, want = hts.residual_norm(x, r, pre=n, gate=full)
    got = full.clone()
    hts.residual_norm(x, r, pre=n, gate=got, out=got)
    assert torch.equal(got, want)
    # no rows
    e, _ = hts.residual_norm(x[:0], r[:0], pre=n)
    assert e.shape == (0, 512)


def test_layer_norm_of_values_far_from_zero():
    # mean 1000, deviation 1: a variance formed as E[x^2] - mean^2 in 32 bits would be off by percents
    g = np.random.default_rng(4)
    r = normal(g, (3, 4096), "f32") + 1000.0
    _, y = hts.residual_norm(None, r, pre=hts.Norm("layer", eps=0.0), out_dtype=torch.float16)
    _, _, want, e = ref.residual_norm(None, f64(r), ("none", 0, None, None), ("layer", 0.0, None, None), None, "none", 1.0)
    assert np.all(np.abs(f64(y) - want) <= 2.0 ** -11 * np.abs(want) + e)
    assert abs(float(f64(y).std()) - 1.0) < 1e-3


def test_norm_keeps_nan_and_infinity_in_their_rows():
    g = np.random.default_rng(5)
    x, r = normal(g, (4, 256), "bf16"), normal(g, (4, 256), "bf16")
    clean, cy = hts.residual_norm(x, r, pre=hts.Norm("rms"))
    x[1, 3], x[2, 200] = float("nan"), float("inf")
    kr, ky = hts.residual_norm(x, r, pre=hts.Norm("rms"))
    for row in (0, 3):
        assert torch.equal(kr[row], clean[row]) and torch.equal(ky[row], cy[row])
    assert bool(torch.isnan(ky[1]).all()) and bool(torch.isnan(ky[2, 200])) and bool(torch.isinf(kr[2, 200]))


# ---- refusals that need tensors on the GPU ---------------------------------

def test_helpers_refuse():
    q, c, table, width = _attn_case(128, 8, 2, 16, "token", "same", [20, 3], "bf16", 9)
    t, n = i32(table)[:, :width], i32([20, 3])
    plan = hts.rope_plan(128, device=DEV)
    k = normal(np.random.default_rng(0), (2, 256), "bf16")
    pos, slots = i32([0, 1]), torch.tensor([0, 1], device=DEV)
    bad = [
        lambda: hts.paged_attn(q[:, :128 * 7], c, t, n),                     # heads not a multiple of the cache's
        lambda: hts.paged_attn(q.float(), c, t, n),
        lambda: hts.paged_attn(q.half(), c, t, n),                           # another 16-bit type than the cache
        lambda: hts.paged_attn(q, c, t, n[:1]),
        lambda: hts.paged_attn(q, c, t.long(), n),
        lambda: hts.paged_attn(q, c, t, n.long()),
        lambda: hts.paged_attn(q, c, t, n.cpu()),
        lambda: hts.paged_attn(q, c, t[:1], n),
        lambda: hts.paged_attn(q, c, t, n, out=q[:, :512]),
        lambda: hts.paged_attn(q, c, t, n, lse=torch.empty((2, 7), device=DEV)),
        lambda: hts.paged_attn(q, c, t, n, window=-1),
        lambda: hts.paged_attn(q.t().contiguous().t(), c, t, n),
        lambda: hts.rope_cache(q, k, k, pos, slots.int(), plan, c),
        lambda: hts.rope_cache(q, k, k[:1], pos, slots, plan, c),
        lambda: hts.rope_cache(q, k[:, :128], k[:, :128], pos, slots, plan, c),
        lambda: hts.rope_cache(q, k, k, pos.long(), slots, plan, c),
        lambda: hts.rope(q, k.half(), pos, plan),
        lambda: hts.rope(q, k, pos[:1], plan),
        lambda: hts.KVCache(c.k, c.v.transpose(1, 2)),
        lambda: hts.KVCache(c.k[:, :, :, ::2], c.v[:, :, :, ::2]),
        lambda: hts.KVCache(c.k.expand(-1, -1, -1, -1)[:1].expand(4, -1, -1, -1), c.v[:1].expand(4, -1, -1, -1)),
        lambda: hts.KVCache(c.k, c.v, k_scale=torch.ones(2, device=DEV)),
        lambda: hts.kv_step(n, n, n, t, 16, -1),
        lambda: hts.kv_step(n, n, n, t, 24, 4),
        lambda: hts.kv_step(n, n.long(), n, t, 16, 4),
        lambda: hts.kv_step(n, i32([1, 1]), i32([0]), t, 16, 4, free_head=n),
        lambda: hts.residual_norm(q, q[:1]),
        lambda: hts.residual_norm(q, q.half()),
        lambda: hts.residual_norm(q, q, pre=hts.Norm("batch")),
        lambda: hts.residual_norm(q, q, pre=hts.Norm("rms", torch.ones(8, device=DEV))),
        lambda: hts.residual_norm(q, q, gate=q.float()),
        lambda: hts.residual_norm(q[:, 1:], q[:, 1:]),
        lambda: hts.residual_norm(q[:, :12], q[:, :12]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(hts.HTSError):
            f()
            say(f"refusal {i} did not happen")


# ---- wide batches, bounds --------------------------------------------------

@pytest.mark.parametrize("B,hq,hk,dim,top", [(130, 2, 1, 64, 1500),      # lengths over several lanes' reach
                                             (64, 4, 2, 128, 700), (65, 3, 3, 8, 900),
                                             (700, 8, 4, 32, 600),
                                             (4500, 2, 2, 16, 560),      # more requests than are split
                                             (2, 800, 800, 8, 1100)])    # more heads than the chip holds at once
def test_paged_attn_of_many_requests(B, hq, hk, dim, top):
    g = np.random.default_rng(B)
    page, pages = 16, 200
    width = -(-top // page)
    c = hts.kv_cache(pages, page, hk, dim, torch.bfloat16, DEV)
    for x in (c.k, c.v):
        x.copy_(torch.randn(x.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(B)).bfloat16())
    lengths = g.integers(0, top + 1, B) * (g.random(B) < 0.8)
    lengths[-1] = top
    table = g.integers(0, pages, (B, width))       # pages are shared: reading them does no harm
    q = normal(g, (B, hq * dim), "bf16")
    lse = torch.empty((B, hq), device=DEV)
    say(f"[attn] B={B} {hq}/{hk} dim={dim} lengths to {top}")
    out = hts.paged_attn(q, c, i32(table), i32(lengths), lse=lse)
    some = np.unique(np.concatenate([g.integers(0, B, 12), [0, B - 1]]))
    heads = np.unique(np.concatenate([g.integers(0, hq, 4), [0, hq - 1]]))
    kv = heads // (hq // hk)
    k, v = f64(c.k[:, :, kv]), f64(c.v[:, :, kv])
    qs = f64(q).reshape(B, hq, dim)[some][:, heads]
    want, wl, err, el = ref.attn(qs, k, v, table[some], lengths[some], page, dim ** -0.5, 0, len(heads))
    got = f64(out).reshape(B, hq, dim)[some][:, heads]
    assert np.all(np.abs(got - want) <= ref.EPS["bf16"] / 2 * np.abs(want) + err + ref.TINY["bf16"])
    gl = f64(lse)[some][:, heads]
    live = ~np.isinf(wl)
    assert np.array_equal(gl[~live], wl[~live]) and np.all(np.abs(gl - wl)[live] <= el[live])


def test_steps_write_only_their_outputs():
    # canary values around the attention's output, sums and workspace, and around the page step's outputs
    pad = 512
    lengths = [3000, 17, 0, 1200]
    q, c, table, width = _attn_case(128, 12, 2, 16, "token", "same", lengths, "bf16", 21)
    need = c.workspace_bytes(4, 12, width, 0)
    assert need > 0
    ws = torch.full((need + 2 * pad,), 0x5A, dtype=torch.uint8, device=DEV)
    o = torch.full((4 * 12 * 128 + 2 * pad,), 9.0, dtype=torch.bfloat16, device=DEV)
    ls = torch.full((48 + 2 * pad,), 9.0, device=DEV)
    lse = ls[pad:-pad].view(4, 12)
    out = hts.paged_attn(q, c, i32(table)[:, :width], i32(lengths), out=o[pad:-pad].view(4, -1), lse=lse,
                         workspace=ws[pad:-pad])
    assert torch.equal(out, hts.paged_attn(q, c, i32(table)[:, :width], i32(lengths)))
    assert torch.all(ws[:pad] == 0x5A) and torch.all(ws[-pad:] == 0x5A)
    for t in (o, ls):
        assert torch.all(t[:pad] == 9.0) and torch.all(t[-pad:] == 9.0)
    B, T = 70, 200
    cached, added, free, tab, _ = _step_case(B, 16, 9, 5, "mixed")
    bufs = {n: torch.full((s + 2 * pad,), -77, dtype=d, device=DEV)
            for n, s, d in (("lengths", B, torch.int32), ("starts", B + 1, torch.int32), ("slots", T, torch.int64),
                            ("positions", T, torch.int32), ("head", 1, torch.int32))}
    st = hts.KVStep(**{n: b[pad:-pad] for n, b in bufs.items()})
    hts.kv_step(i32(cached), i32(added), i32(free), i32(tab)[:, :9], 16, T, out=st)
    for n, b in bufs.items():
        assert torch.all(b[:pad] == -77) and torch.all(b[-pad:] == -77), n
        assert torch.all(b[pad:-pad] != -77), n


def test_debug_mode_refuses_short_buffers(monkeypatch):
    # HTS_DEBUG=1 finds a buffer shorter than the call needs before anything is enqueued, and changes no result
    from test_gpu_debug import DeviceBuffer
    lengths = [900, 3]
    q, c, table, width = _attn_case(128, 8, 2, 16, "token", "same", lengths, "bf16", 31)
    t, n = i32(table)[:, :width], i32(lengths)
    plain = hts.paged_attn(q, c, t, n)
    x = normal(np.random.default_rng(0), (64, 4096), "bf16")
    r0, y0 = hts.residual_norm(x, x, pre=hts.Norm("rms"))
    monkeypatch.setenv("HTS_DEBUG", "1")
    assert torch.equal(hts.paged_attn(q, c, t, n), plain)
    r1, y1 = hts.residual_norm(x, x, pre=hts.Norm("rms"))
    assert torch.equal(r0, r1) and torch.equal(y0, y1)
    short = DeviceBuffer(64 * 4096)               # half of a 64 x 4096 matrix of 16-bit values
    big = torch.empty((2048, 16, 2, 128), dtype=torch.bfloat16, device=DEV)
    import ctypes
    L = hts.lib()
    try:
        d = hts.hts_norm_desc(1, 1, 0, 1, 1e-6, 1e-6, 1.0, 0)
        assert L.hts_residual_norm(ctypes.byref(d), 64, 4096, x.data_ptr(), 4096, None, None, None, 0, None, 0, None, None,
                                   None, 0, short.ptr.value, 4096, None) == 3
        assert b"Y needs" in L.hts_last_error()
        kv = hts.KVCache(big, big.clone())
        assert L.hts_paged_attn(1, 2, 8, ctypes.byref(kv.desc), q.data_ptr(), 1024, short.ptr.value, kv.v.data_ptr(), None,
                                None, t.data_ptr(), t.stride(0), width, n.data_ptr(), 0.1, 0, plain.data_ptr(), 1024, None,
                                None, 0, None) == 3
        assert b"k_cache needs" in L.hts_last_error()
    finally:
        short.free()


def test_two_attention_calls_at_once():
    # split calls on two streams, each with a workspace of its own, many times over
    a = _attn_case(128, 16, 2, 16, "token", "same", [9000, 70, 0], "bf16", 41)
    b = _attn_case(128, 8, 8, 64, "head", "fp8", [3000, 1, 777, 5000], "bf16", 42)
    calls = [(q, c, i32(t)[:, :w].contiguous(), i32(n)) for (q, c, t, w), n in ((a, [9000, 70, 0]), (b, [3000, 1, 777, 5000]))]
    want = [hts.paged_attn(*x) for x in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for k in (0, 1):
            got[k].append(hts.paged_attn(*calls[k], stream=streams[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(torch.equal(x, want[k]) for x in got[k])


def test_one_page_for_all_and_for_a_whole_row():
    # the same page many times in a row of the table, and the same row for every request
    c = hts.kv_cache(2, 16, 2, 64, torch.float16, DEV)
    g = np.random.default_rng(3)
    c.k.copy_(normal(g, c.k.shape, "f16"))
    c.v.copy_(normal(g, c.v.shape, "f16"))
    q = normal(g, (1, 4 * 64), "f16").expand(3, -1).contiguous()
    table = np.full((3, 80), 1)
    lengths = [1280, 16, 1279]
    out = hts.paged_attn(q, c, i32(table), i32(lengths))
    _check_attn(q, c, table, 80, lengths, 4, 0, 64 ** -0.5, out, None, "f16")
    # 1280 tokens that repeat 16 tokens 80 times: the attention over the 16
    assert float((out[0].float() - out[1].float()).abs().max()) <= 2.0 ** -10 * float(c.v.float().abs().max())


@pytest.mark.parametrize("M", [1, 5])
def test_functions_with_the_c_names_match_the_helpers(M):
    # the marshalling under the entry points' own names; one row may come as a view with any stride between rows
    g = np.random.default_rng(M)
    dim, hq, hk, page, width = 64, 4, 2, 16, 3

    def view(cols):
        x = normal(g, (M, cols), "bf16")
        return x if M > 1 else torch.as_strided(x, (1, cols), (cols + 3, 1))
    i64 = dict(dtype=torch.int64, device=DEV)
    # page step
    cached, added, free = i32(g.integers(0, 20, M)), i32(np.ones(M)), i32(g.permutation(32))
    tables = [torch.full((M, width), 31, dtype=torch.int32, device=DEV) for _ in range(2)]
    want = hts.kv_step(cached, added, free, tables[0], page, M + 2, free_head=i32([1]))
    got = hts.KVStep(*(torch.empty_like(x) for x in (want.lengths, want.starts, want.slots, want.positions, want.head)))
    hts.hts_kv_step(cached, added, page, free, i32([1]), tables[1] if M > 1 else tables[1].as_strided((1, width), (1, 1)), got.lengths,
                    got.starts, got.slots, got.positions, got.head)
    for name in ("lengths", "starts", "slots", "positions", "head"):
        assert torch.equal(getattr(got, name), getattr(want, name)), name
    assert torch.equal(*tables)
    # rotary
    plan = hts.rope_plan(dim, 32, layout="interleaved", magnitude=1.5, device=DEV)
    turns = hts.hts_rope_plan(hts.hts_rope_scaling(32, 0, 10000.0, 1.0, 0.0, 1.0, 32.0))
    assert np.array_equal(turns, plan.turns.cpu().numpy())
    desc = hts.hts_rope_desc(hts.HTS_BF16, plan.layout, dim, 32, hq, hk, 1.5, 0)
    q, k, v = view(hq * dim), view(hk * dim), view(hk * dim)
    pos, slots = i32(np.arange(M) * 7 + 3), torch.tensor(g.permutation(64)[:M], **i64)
    outs = [torch.zeros((M, h * dim), dtype=torch.bfloat16, device=DEV) for h in (hq, hk, hq, hk)]
    hts.rope(q, k, pos, plan, q_out=outs[0], k_out=outs[1])
    hts.hts_rope(desc, plan.turns, pos, q, outs[2], k, outs[3])
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3]) and bool((outs[1] != 0).any())
    caches = [hts.kv_cache(4, page, hk, dim, torch.bfloat16, DEV) for _ in range(3)]
    hts.rope_cache(q, k, v, pos, slots, plan, caches[0], q_out=outs[0])
    hts.hts_rope_cache(desc, plan.turns, pos, slots, q, outs[2], k, v, caches[1].desc, caches[1].k, caches[1].v)
    starts = torch.arange(M + 1, dtype=torch.int32, device=DEV)
    hts.hts_rope_cache_rows(desc, plan.turns, starts, pos, slots, q, outs[1].new_empty((M, hq * dim)), k, v, caches[2].desc, caches[2].k,
                            caches[2].v)
    for c in caches[1:]:
        assert torch.equal(c.k, caches[0].k) and torch.equal(c.v, caches[0].v)
    assert torch.equal(outs[0], outs[2]) and bool((caches[0].v != 0).any())
    # attention
    cache, table, n = caches[0], i32(g.integers(0, 4, (M, width))), i32(g.integers(1, 48, M))
    lse = [torch.empty((M, hq), device=DEV) for _ in range(2)]
    want = hts.paged_attn(q, cache, table, n, scale=0.2, window=20, lse=lse[0])
    hts.hts_paged_attn(hq, cache.desc, q, cache.k, cache.v, table, n, 0.2, outs[2], window=20, lse=lse[1])
    assert torch.equal(outs[2], want) and torch.equal(*lse)
    # norm: gates of a row per token and of one row
    x, r, w = view(256), normal(g, (M, 256), "f32"), normal(g, (256,), "bf16")
    d = hts.hts_norm_desc(hts.HTS_BF16, hts.HTS_F32, 0, 1, 0.0, 1e-5, 0.5, 1)
    for gate in (view(256), normal(g, (256,), "bf16")):
        want = hts.residual_norm(x, r, pre=hts.Norm("rms", w, eps=1e-5), gate=gate, gate_act="sigmoid", scale=0.5)
        got = [torch.empty_like(r), torch.empty((M, 256), dtype=torch.bfloat16, device=DEV)]
        hts.hts_residual_norm(d, M, 256, x, None, None, gate, r, w, None, *got)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
