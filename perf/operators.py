"""Cases of the serving operators around the hybrid products: what one decode (or prefill) step of a
decoder block needs besides its projections.

  step   block tables, slot maps and positions built on the GPU from request lengths
  rope   rotary positions on q and k, with k and v written into the paged key-value cache
  attn   attention of one new token per request over the paged cache
  norm   norm after a block, gate, residual scale and add, norm before the next block

``run`` computes an operator in elementary torch operations (32-bit arithmetic, 64-bit angles), or,
with ``own`` set, calls the library.  Shapes are those of the 7B / 13B layers the repository measures
(hidden 4096 / 5120, heads of 128) or generic ones.
"""
import math

import torch

own = False

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "fp8": 1}


def listed():
    return [
        # one scheduler tick of a small decode batch: every request adds one token; pure latency
        dict(name="step decode 64", op="step", requests=64, context=2048, added=1, page=16),
        # a tick that admits many prompts beside running requests (chunked prefill of up to 2048 tokens each)
        dict(name="step mixed 512", op="step", requests=512, context=16384, added=2048, page=16),
        # a single chat's next token on a 7B block: 32 heads, no sharing
        dict(name="rope one token", op="rope", tokens=1, hq=32, hk=32, dim=128, rot=128, layout="half", rule="plain",
             factor=1.0, reach=4096, page=16, order="token", dtype="bf16"),
        # a decode batch padded to its captured size (13B heads, shared), part of the head, pairs side by side
        dict(name="rope batch 61", op="rope", tokens=61, hq=40, hk=8, dim=128, rot=64, layout="interleaved",
             rule="linear", factor=4.0, reach=32768, page=64, order="head", dtype="f16"),
        # a long prompt's prefill with positions scaled past the trained context
        dict(name="rope prefill 8192", op="rope", tokens=8192, hq=32, hk=32, dim=128, rot=128, layout="half",
             rule="ramp", factor=8.0, reach=1000000, page=16, order="token", dtype="bf16"),
        # a single short chat: the smallest attention call, latency only
        dict(name="attn one short", op="attn", requests=1, most=200, hq=32, hk=32, dim=128, page=16, order="token",
             dtype="bf16", cache="bf16", window=0),
        # an ordinary serving batch: ragged lengths, four query heads to a cache head
        dict(name="attn batch 32", op="attn", requests=32, most=4096, hq=32, hk=8, dim=128, page=16, order="token",
             dtype="f16", cache="f16", window=0),
        # a larger batch on an 8-bit cache, five query heads to a cache head
        dict(name="attn 8-bit 64", op="attn", requests=64, most=8191, hq=40, hk=8, dim=128, page=64, order="head",
             dtype="bf16", cache="fp8", window=0),
        # few very long documents: the length is split over the chip and joined
        dict(name="attn long 4", op="attn", requests=4, most=131072, hq=64, hk=8, dim=128, page=32, order="token",
             dtype="bf16", cache="bf16", window=0),
        # one token of a 7B block: residual add and the next norm
        dict(name="norm one token", op="norm", rows=1, width=4096, post="none", pre="rms", gate="none", act="none",
             scale=1.0, dtype="bf16", rdtype="bf16"),
        # a 13B block with norms on both sides, a learned gate per channel, a residual stream in 32 bits
        dict(name="norm both 300", op="norm", rows=300, width=5120, post="rms", pre="rms", gate="channel", act="none",
             scale=0.5, dtype="f16", rdtype="f32"),
        # a large prefill batch, layer norms, a gate computed from the token
        dict(name="norm gated 16384", op="norm", rows=16384, width=4096, post="layer", pre="layer", gate="token",
             act="sigmoid", scale=1.0, dtype="bf16", rdtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "rope", "attn", "attn", "norm"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "step":
        return dict(op=op, requests=_log(rng, 1, 512), context=_log(rng, 16, 16384),
                    added=rng.choice([1, 1, _log(rng, 2, 2048)]), page=page)
    dtype = rng.choice(["bf16", "f16"])
    hk = rng.choice([1, 2, 3, 4, 5, 8, 10])
    group = min(rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16, 20]), 64 // hk)
    order = rng.choice(["token", "head"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        rot = rng.choice([dim, dim, dim // 2, 16])
        most = 8192 * 32 * 128 * 3 // ((hk * group + 2 * hk) * dim)
        return dict(op=op, tokens=_log(rng, 1, min(8192, most)), hq=hk * group, hk=hk, dim=dim, rot=rot,
                    layout=rng.choice(["half", "interleaved"]), rule=rng.choice(["plain", "linear", "base", "ramp"]),
                    factor=rng.choice([1.0, 2.0, 5.5, 16.0]), reach=_log(rng, 64, 1000000), page=page, order=order,
                    dtype=dtype)
    if op == "attn":
        dim = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
        cache = rng.choice([dtype, dtype, "fp8"])
        requests = _log(rng, 1, 256)
        most = 4 * 131072 * 8 * 128 // (requests * hk * dim)
        return dict(op=op, requests=requests, most=_log(rng, 1, max(1, min(131072, most))), hq=hk * group, hk=hk,
                    dim=dim, page=page, order=order, dtype=dtype, cache=cache,
                    window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]))
    width = 8 * _log(rng, 8, 2048)
    rows = _log(rng, 1, max(1, min(65536, 16384 * 4096 // width // 2)))
    post, pre = rng.choice([("none", "rms"), ("rms", "rms"), ("layer", "layer"), ("rms", "none"), ("none", "layer")])
    return dict(op=op, rows=rows, width=width, post=post, pre=pre, gate=rng.choice(["none", "channel", "token"]),
                act=rng.choice(["none", "sigmoid", "silu"]), scale=rng.choice([1.0, 0.25, 1.7]), dtype=dtype,
                rdtype=rng.choice([dtype, "f32"]))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _lengths(case):
    """The batch's lengths: evenly spread from short to the longest, so that a batch is ragged; in a batch
    of eight and more the first is a padding row without tokens."""
    n, most = case["requests"], case["most"]
    got = [max(1, (i + 1) * most // n) for i in range(n)]
    if n >= 8:
        got[0] = 0
    return got


def _step_sizes(case):
    n = case["requests"]
    cached = [(i * 7919 % n) * case["context"] // max(1, n) for i in range(n)]
    if case["added"] == 1:
        return cached, [1] * n
    return cached, [1 if i % 4 else 1 + (i * 104729 % n) * (case["added"] - 1) // max(1, n - 1) for i in range(n)]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, sigma=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * sigma).to(DT[dtype])


def _big_normal(g, shape, dtype):
    """Normal values for a large cache, made in 16 bits (8-bit ones by way of 32 in slices of the first axis)."""
    if dtype != "fp8":
        return torch.randn(shape, generator=g, device=DEV, dtype=DT[dtype])
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float16).to(DT["fp8"])


def _cache_view(t, order):
    """[pages, page, heads, dim] over storage in that order, or with the heads outside the page's tokens."""
    return t if order == "token" else t.transpose(1, 2)


def _storage(pages, page, heads, dim, order):
    return (pages, page, heads, dim) if order == "token" else (pages, heads, page, dim)


def prepare(case, seed):
    return {"step": _prepare_step, "rope": _prepare_rope, "attn": _prepare_attn, "norm": _prepare_norm}[case["op"]](
        case, seed)


def _prepare_step(case, seed):
    g = _gen(seed)
    cached, added = _step_sizes(case)
    n, page = case["requests"], case["page"]
    order = torch.randperm(n, generator=g, device=DEV)
    cached = torch.tensor(cached, dtype=torch.int32, device=DEV)[order].contiguous()
    added = torch.tensor(added, dtype=torch.int32, device=DEV)[order].contiguous()
    width = -(-(case["context"] + case["added"]) // page)
    pages = n * width
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    have = (cached + page - 1) // page
    table = ids.view(n, width).clone()                        # the pages that running requests hold
    table[torch.arange(width, device=DEV)[None] >= have[:, None]] = -1
    free = ids.view(n, width)[torch.arange(width, device=DEV)[None] >= have[:, None]].contiguous()
    tokens = int(sum(_step_sizes(case)[1]))
    return dict(case=case, cached=cached, added=added, table=table, free=free, page=page,
                tokens=tokens + tokens % 7, head=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_rope(case, seed):
    g = _gen(seed)
    T, hq, hk, dim, page = (case[k] for k in ("tokens", "hq", "hk", "dim", "page"))
    # q, k and v lie side by side in the rows of one projection's output
    qkv = _normal(g, (T, (hq + 2 * hk) * dim), case["dtype"])
    q, k, v = qkv[:, :hq * dim], qkv[:, hq * dim:(hq + hk) * dim], qkv[:, (hq + hk) * dim:]
    pages = -(-T // page) + 3
    if T < 256:                                               # a token each of as many requests
        slots = torch.randperm(pages * page, generator=g, device=DEV)[:T].contiguous()
        positions = torch.randint(0, case["reach"], (T,), generator=g, device=DEV, dtype=torch.int32)
    else:                                                     # prompts: runs of up to 2048 tokens, page after page
        t = torch.arange(T, device=DEV)
        slots = torch.randperm(pages, generator=g, device=DEV)[t // page] * page + t % page
        begin = torch.randint(0, case["reach"], (T // 2048 + 1,), generator=g, device=DEV)
        positions = (begin[t // 2048] + t % 2048).int()
    if T >= 16:                                               # the batch's padding
        positions[T - T // 16:] = -1
        slots[T - T // 16:] = -1
    kc = _cache_view(_normal(g, _storage(pages, page, hk, dim, case["order"]), case["dtype"]), case["order"])
    vc = _cache_view(_normal(g, _storage(pages, page, hk, dim, case["order"]), case["dtype"]), case["order"])
    s = dict(case=case, q=q, k=k, v=v, positions=positions, slots=slots, kc=kc, vc=vc,
             q_out=torch.zeros((T, hq * dim), dtype=DT[case["dtype"]], device=DEV),
             freq=torch.tensor(_frequencies(case), dtype=torch.float64, device=DEV))
    if own:
        import tile_gemm_amd as hts
        s["plan"] = hts.rope_plan(dim, case["rot"], theta=10000.0, layout=case["layout"], rule=case["rule"],
                                  factor=case["factor"], context=4096, low=1.0, high=32.0, device=DEV)
        s["cache"] = hts.KVCache(kc, vc)
    return s


def _frequencies(case):
    """Radians per position of each pair, in 64 bits: theta^(-2i/R), and its scaling for long contexts."""
    R, s, theta = case["rot"], case["factor"], 10000.0
    if case["rule"] == "base":
        theta *= s ** (R / (R - 2))
    f = [theta ** (-2.0 * i / R) for i in range(R // 2)]
    if case["rule"] == "linear":
        f = [x / s for x in f]
    if case["rule"] == "ramp":                                # pairs with few turns over the context are stretched
        keep = [min(1.0, max(0.0, (4096 * x / (2 * math.pi) - 1.0) / 31.0)) for x in f]
        f = [x * (c + (1.0 - c) / s) for x, c in zip(f, keep)]
    return f


def _prepare_attn(case, seed):
    g = _gen(seed)
    B, hq, hk, dim, page = (case[k] for k in ("requests", "hq", "hk", "dim", "page"))
    lengths = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
    lengths = lengths[torch.randperm(B, generator=g, device=DEV)].contiguous()
    used = (lengths + page - 1) // page
    width = -(-case["most"] // page)
    total = int(sum(-(-x // page) for x in _lengths(case)))
    pages = total + 2
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(width, device=DEV)[None] < used[:, None]] = ids[:total]
    shape = _storage(pages, page, hk, dim, case["order"])
    kc = _cache_view(_big_normal(g, shape, case["cache"]), case["order"])
    vc = _cache_view(_big_normal(g, shape, case["cache"]), case["order"])
    s = dict(case=case, q=_normal(g, (B, hq * dim), case["dtype"]), kc=kc, vc=vc, table=table, lengths=lengths,
             ks=None, vs=None)
    if case["cache"] == "fp8":
        s["ks"] = torch.rand(hk, generator=g, device=DEV) + 0.5
        s["vs"] = torch.rand(hk, generator=g, device=DEV) + 0.5
    if own:
        import tile_gemm_amd as hts
        s["cache"] = hts.KVCache(kc, vc, k_scale=s["ks"], v_scale=s["vs"])
    return s


def _prepare_norm(case, seed):
    g = _gen(seed)
    M, N, dt = case["rows"], case["width"], case["dtype"]
    s = dict(case=case, block=_normal(g, (M, N), dt), residual=_normal(g, (M, N), case["rdtype"], 2.0), gate=None)
    if case["gate"] == "channel":
        s["gate"] = _normal(g, (N,), dt)
    elif case["gate"] == "token":
        s["gate"] = _normal(g, (M, N), dt)
    for side in ("post", "pre"):
        s[side + "_w"] = _normal(g, (N,), dt, 0.1) + 1.0 if case[side] != "none" else None
        s[side + "_b"] = _normal(g, (N,), dt, 0.1) if case[side] == "layer" else None
        if own and case[side] != "none":
            import tile_gemm_amd as hts
            s[side] = hts.Norm(case[side], s[side + "_w"], s[side + "_b"], eps=1e-5)
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"step": _own_step, "rope": _own_rope, "attn": _own_attn, "norm": _own_norm}[op](s)
    return {"step": _plain_step, "rope": _plain_rope, "attn": _plain_attn, "norm": _plain_norm}[op](s)


def _own_step(s):
    import tile_gemm_amd as hts
    st = hts.kv_step(s["cached"], s["added"], s["free"], s["table"], s["page"], s["tokens"], free_head=s["head"])
    return dict(table=s["table"], lengths=st.lengths, starts=st.starts, slots=st.slots, positions=st.positions,
                head=st.head)


def _own_rope(s):
    import tile_gemm_amd as hts
    hts.rope_cache(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["plan"], s["cache"], q_out=s["q_out"])
    return dict(q=s["q_out"], k_cache=s["kc"], v_cache=s["vc"])


def _own_attn(s):
    import tile_gemm_amd as hts
    c = s["case"]
    lse = torch.empty((c["requests"], c["hq"]), dtype=torch.float32, device=DEV)
    out = hts.paged_attn(s["q"], s["cache"], s["table"], s["lengths"], scale=c["dim"] ** -0.5, window=c["window"],
                         lse=lse)
    return dict(out=out, lse=lse)


def _own_norm(s):
    import tile_gemm_amd as hts
    c = s["case"]
    r, y = hts.residual_norm(s["block"], s["residual"], post=s.get("post"), pre=s.get("pre"), gate=s["gate"],
                             gate_act=c["act"], scale=c["scale"])
    return dict(residual=r) if y is None else dict(residual=r, out=y)


def _plain_step(s):
    page, table, free, T = s["page"], s["table"], s["free"], s["tokens"]
    n, width = table.shape
    cached, added = s["cached"].long(), s["added"].long()
    ends = added.cumsum(0)
    starts = torch.cat([ends.new_zeros(1), ends])
    lengths = (cached + added).clamp(max=width * page)
    have, want = (cached + page - 1) // page, (lengths + page - 1) // page
    new = want - have
    base = s["head"].long() + new.cumsum(0) - new
    col = torch.arange(width, device=table.device)[None]
    take = (base - have)[:, None] + col
    got = torch.where(take < free.numel(), free[take.clamp(0, max(0, free.numel() - 1))], -1)
    table.copy_(torch.where((col >= have[:, None]) & (col < want[:, None]), got, table))
    t = torch.arange(T, device=table.device)
    who = torch.searchsorted(ends, t, right=True).clamp(max=n - 1)
    position = cached[who] + t - starts[who]
    held = table[who, (position // page).clamp(0, width - 1)].long()
    slot = torch.where((held >= 0) & (position < width * page), held * page + position % page, -1)
    live = t < ends[-1]
    return dict(table=table, lengths=lengths.int(), starts=starts.int(), slots=torch.where(live, slot, -1),
                positions=torch.where(live, position, -1).int(), head=(s["head"] + new.sum()).int())


def _rotate(x, cos, sin, R, layout):
    """x [T, heads, dim] in 32 bits, its first R entries of each head turned by the angles of cos, sin [T, 1, R/2]."""
    if layout == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, x[..., R:]], -1)
    a, b = x[..., 0:R:2], x[..., 1:R:2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), x[..., R:]], -1)


def _plain_rope(s):
    c = s["case"]
    T, dim, page = c["tokens"], c["dim"], c["page"]
    angle = s["positions"].double()[:, None] * s["freq"][None]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _rotate(s["q"].float().view(T, c["hq"], dim), cos, sin, c["rot"], c["layout"]).to(s["q"].dtype)
    k = _rotate(s["k"].float().view(T, c["hk"], dim), cos, sin, c["rot"], c["layout"]).to(s["k"].dtype)
    q = torch.where(s["positions"][:, None] >= 0, q.view(T, -1), s["q_out"])
    # the padding behind the last token writes the first token again
    src = torch.where(s["slots"] >= 0, torch.arange(T, device=q.device), 0)
    slots = s["slots"][src]
    s["kc"][slots // page, slots % page] = k[src]
    s["vc"][slots // page, slots % page] = s["v"].view(T, c["hk"], dim)[src]
    return dict(q=q, k_cache=s["kc"], v_cache=s["vc"])


def _values(cache, ids, scale):
    """The gathered pages [B, tokens, heads, dim] in 32 bits, heads in front of tokens."""
    if cache.dtype == torch.float8_e4m3fn:
        got = cache.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
    else:
        got = cache[ids].float()
    got = got.flatten(1, 2)
    if scale is not None:
        got = got * scale[:, None]
    return got.transpose(1, 2)


def _plain_attn(s):
    c = s["case"]
    B, hq, hk, dim = c["requests"], c["hq"], c["hk"], c["dim"]
    ids = s["table"].long().clamp(0)
    k, v = _values(s["kc"], ids, s["ks"]), _values(s["vc"], ids, s["vs"])
    q = s["q"].float().view(B, hk, hq // hk, dim)
    score = torch.matmul(q, k.transpose(2, 3)) * (dim ** -0.5)
    at = torch.arange(score.shape[3], device=score.device)[None]
    length = s["lengths"].long()[:, None]
    keep = at < length
    if c["window"]:
        keep = keep & (at >= length - c["window"])
    score = score.masked_fill(~keep[:, None, None], -math.inf)
    top = score.amax(3, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(3, keepdim=True)
    out = torch.where(total > 0, torch.matmul(p, v) / total, 0.0)
    return dict(out=out.reshape(B, hq * dim).to(s["q"].dtype), lse=(top + total.log()).view(B, hq))


def _norm(x, kind, w, b):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-5) * w.float()
    return x if b is None else x + b.float()


def _plain_norm(s):
    c = s["case"]
    b = _norm(s["block"].float(), c["post"], s["post_w"], s["post_b"])
    if s["gate"] is not None:
        g = s["gate"].float()
        if c["act"] != "none":
            g = 1.0 / (1.0 + torch.exp(-g)) * (g if c["act"] == "silu" else 1.0)
        b = b * g
    r = s["residual"].float() + c["scale"] * b
    got = dict(residual=r.to(s["residual"].dtype))
    if c["pre"] != "none":
        got["out"] = _norm(r, c["pre"], s["pre_w"], s["pre_b"]).to(s["block"].dtype)
    return got


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without, and the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "step":
        cached, added = _step_sizes(case)
        page, tokens = case["page"], sum(added)
        new = sum(-(-(c + a) // page) - -(-c // page) for c, a in zip(cached, added))
        return dict(bytes=16 * case["requests"] + 8 * new + 12 * tokens, flops=0)
    if op == "rope":
        live = case["tokens"] - (case["tokens"] // 16 if case["tokens"] >= 16 else 0)
        n = (case["hq"] + 2 * case["hk"]) * case["dim"]
        return dict(bytes=live * (2 * n * SIZE[case["dtype"]] + 12),
                    flops=3 * live * (case["hq"] + case["hk"]) * case["rot"])
    if op == "attn":
        live = sum(min(x, case["window"]) if case["window"] else x for x in _lengths(case))
        io = case["requests"] * case["hq"] * (2 * case["dim"] * SIZE[case["dtype"]] + 4)
        return dict(bytes=2 * live * case["hk"] * case["dim"] * SIZE[case["cache"]] + io,
                    flops=4 * live * case["hq"] * case["dim"])
    n = case["rows"] * case["width"]
    each = SIZE[case["dtype"]] * (1 + (case["pre"] != "none") + (case["gate"] == "token")) + 2 * SIZE[case["rdtype"]]
    return dict(bytes=n * each, flops=10 * n)


def exact(case, seed):
    s = prepare(case, seed)
    return {"step": _exact_step, "rope": _exact_rope, "attn": _exact_attn, "norm": _exact_norm}[case["op"]](case, s)


def _exact_step(case, s):
    page, T = s["page"], s["tokens"]
    cached, added, free, table = (s[k].tolist() for k in ("cached", "added", "free", "table"))
    starts, lengths, slots, positions, head = [0], [], [], [], int(s["head"])
    for row, c, a in zip(table, cached, added):
        n = min(c + a, len(row) * page)
        for j in range(-(-c // page), -(-n // page)):
            row[j] = free[head] if head < len(free) else -1
            head += 1
        for p in range(c, c + a):
            held = row[p // page] if p < len(row) * page else -1
            slots.append(held * page + p % page if held >= 0 else -1)
            positions.append(p)
        lengths.append(n)
        starts.append(starts[-1] + a)
    pad = [-1] * (T - len(slots))
    to = lambda v, dt: torch.tensor(v, dtype=dt, device=DEV)  # noqa: E731
    return dict(table=to(table, torch.int32), lengths=to(lengths, torch.int32), starts=to(starts, torch.int32),
                slots=to(slots + pad, torch.int64), positions=to(positions + pad, torch.int32),
                head=to([head], torch.int32))


def _exact_rope(case, s):
    R, dim = case["rot"], case["dim"]
    # a turn by the angle, as a product of complex numbers
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s["positions"].double()[:, None] * s["freq"])

    def turned(x, heads):
        x = x.double().reshape(case["tokens"], heads, dim).clone()
        pairs = x[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2) if case["layout"] == "half" \
            else x[..., :R].unflatten(-1, (R // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
        x[..., :R] = (z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2)
        return x

    q, kc, vc = s["q_out"].double(), s["kc"].double(), s["vc"].double()
    live = s["positions"] >= 0
    q[live] = turned(s["q"], case["hq"]).flatten(1)[live]
    at = s["slots"][s["slots"] >= 0]
    where = (torch.div(at, case["page"], rounding_mode="floor"), at.remainder(case["page"]))
    kc[where] = turned(s["k"], case["hk"])[s["slots"] >= 0]
    vc[where] = s["v"].double().reshape(case["tokens"], case["hk"], dim)[s["slots"] >= 0]
    return dict(q=q, k_cache=kc, v_cache=vc)


def _exact_attn(case, s):
    B, hq, hk, dim, page = (case[k] for k in ("requests", "hq", "hk", "dim", "page"))
    out = torch.zeros((B, hq, dim), dtype=torch.float64, device=DEV)
    lse = torch.full((B, hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lengths"].tolist()):
        if n == 0:
            continue
        first = max(0, n - case["window"]) if case["window"] else 0
        t = torch.arange(first, n, device=DEV)
        rows = s["table"][b].long()[t // page]
        for h in range(hk):
            k = s["kc"][:, :, h].view(torch.uint8)[rows, t % page].view(s["kc"].dtype).double()
            v = s["vc"][:, :, h].view(torch.uint8)[rows, t % page].view(s["vc"].dtype).double()
            if s["ks"] is not None:
                k, v = k * s["ks"][h].double(), v * s["vs"][h].double()
            heads = slice(h * (hq // hk), (h + 1) * (hq // hk))
            score = (s["q"][b].double().view(hq, dim)[heads] @ k.T) / math.sqrt(dim)
            lse[b, heads] = torch.logsumexp(score, 1)
            out[b, heads] = torch.exp(score - lse[b, heads][:, None]) @ v
    return dict(out=out.view(B, hq * dim), lse=lse)


def _exact_norm(case, s):
    def normed(x, side):
        if case[side] == "none":
            return x
        if case[side] == "layer":
            var, mean = torch.var_mean(x, 1, keepdim=True, correction=0)
            x = (x - mean) / torch.sqrt(var + 1e-5) * s[side + "_w"].double()
            return x + s[side + "_b"].double()
        return x / torch.sqrt(x.square().sum(1, keepdim=True) / x.shape[1] + 1e-5) * s[side + "_w"].double()

    b = normed(s["block"].double(), "post")
    if s["gate"] is not None:
        g = s["gate"].double()
        b = b * {"none": g, "sigmoid": torch.sigmoid(g), "silu": g * torch.sigmoid(g)}[case["act"]]
    r = s["residual"].double() + case["scale"] * b
    return dict(residual=r) if case["pre"] == "none" else dict(residual=r, out=normed(r, "pre"))
