"""Tensor-level helpers of the steps around a decoder block's products.

    step = kv_step(cached, added, free_pages, table, page, tokens)       pages, slots and positions
    rope_cache(q, k, v, step.positions, step.slots, plan, cache)         rotary positions, k and v cached
    a = paged_attn(q, cache, table, step.lengths, scale)                 one new token per request
    x, y = residual_norm(block_out, x, post=..., pre=..., gate=...)      between two blocks

As in the rest of the package these only check and marshal arguments; the work is in the HIP kernels.
Matrices are [tokens, heads * head size] with any leading dimension, as the products write them.  All
tensors of a call live on one GPU; the call runs on ``stream`` (default: that GPU's current stream), and
what it allocates belongs to that stream.  Nothing here reads device memory on the host, so every call can
be captured in a HIP graph (give ``out`` buffers there, or keep the ones returned at capture).
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
from typing import Optional

import torch

import tile_gemm_amd as _c

_LAYOUTS = {"half": 0, "interleaved": 1}
_RULES = {"plain": 0, "linear": 1, "base": 2, "ramp": 3, "ramp_pairs": 4}
_NORMS = {"none": 0, "rms": 1, "layer": 2}
_GATES = {"none": 0, "sigmoid": 1, "silu": 2}
_16 = (torch.float16, torch.bfloat16)


def _bad(text: str, status: int = 1):
    raise _c.HTSError(status, text)


def _choice(table: dict, key, what: str) -> int:
    if key not in table:
        _bad(f"{what} {key!r} is not one of {', '.join(table)}")
    return table[key]


def _explain(t, name: str, rows, cols, dtypes, dev: int):
    """Say what is wrong with a tensor that a check below has refused."""
    if t.get_device() != dev:
        _bad(f"{name} is on {t.device}, expected GPU {dev}" if dev >= 0 else f"{name} must be on a GPU, not on {t.device}")
    if t.dtype not in dtypes:
        _bad(f"{name} has type {t.dtype}, expected {' or '.join(map(str, dtypes))}", 2)
    want = (rows,) if cols is None else (rows, cols)
    if tuple(t.shape) != want:
        _bad(f"{name} has shape {tuple(t.shape)}, expected {want}", 3)
    _bad(f"{name} must be contiguous along its rows", 3)


def _gpu(t: torch.Tensor, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        _bad(f"{name} must be on a GPU, not on {t.device}")
    return dev


def _lead(t: torch.Tensor, name: str, rows: int, cols: int, dtype, dev: int) -> int:
    """Leading dimension of a [rows, cols] matrix of this type on this GPU (a matrix of one row may carry any
    stride there: it gets one that the library takes)."""
    if t.dtype is dtype and t.get_device() == dev and t.dim() == 2:
        r, c = t.shape
        if r == rows and c == cols:
            lead, one = t.stride()
            if one == 1 or cols <= 1 or rows == 0:
                return lead if rows > 1 else (cols + 7) // 8 * 8
    return _explain(t, name, rows, cols, (dtype,), dev)


def _vec(t: torch.Tensor, name: str, n: int, dtype, dev: int) -> int:
    """Address of a contiguous vector of n entries of this type on this GPU."""
    if t.dtype is dtype and t.get_device() == dev and t.dim() == 1 and t.shape[0] == n and (n <= 1 or t.stride(0) == 1):
        return t.data_ptr()
    return _explain(t, name, n, None, (dtype,), dev)


def _table(t: torch.Tensor, rows: int, dev: int) -> int:
    """Leading dimension of a block table int32 [rows, width]."""
    if t.dim() != 2:
        _bad("block_table must be [requests, pages of a request]", 3)
    width = t.shape[1]
    _lead(t, "block_table", rows, width, torch.int32, dev)
    return t.stride(0) if rows > 1 else width


@contextlib.contextmanager
def _switched(dev, stream):
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            s = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=dev)
            if s.device_index != dev:
                _bad(f"the stream belongs to GPU {s.device_index}, the tensors to GPU {dev}")
            with torch.cuda.stream(s):
                yield


_STAY = contextlib.nullcontext()


def _scope(dev: int, stream):
    """Make the tensors' GPU and the call's stream current, for the launch and for what it allocates."""
    if stream is None and torch.cuda.current_device() == dev:
        return _STAY
    return _switched(dev, stream)


# --------------------------------------------------------------------------
# pages of the key-value cache
# --------------------------------------------------------------------------

class KVCache:
    """A paged key-value cache: k and v as [pages, page, heads, head size] tensors (or views) of one shape
    and one set of strides, entries of a head consecutive.  An 8-bit (float8_e4m3fn) cache holds
    value / scale with one float32 scale per head (none: 1)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            _bad("k and v must be [pages, page, heads, head size] tensors of one shape and type", 3)
        if k.dtype not in _16 + (torch.float8_e4m3fn,):
            _bad(f"a cache of type {k.dtype}", 2)
        used = [i for i in range(3) if k.shape[i] > 1]
        if any(k.stride(i) != v.stride(i) for i in used) or k.stride(3) != 1 or v.stride(3) != 1:
            _bad("k and v must have one set of strides, with the entries of a head consecutive", 3)
        dev = _gpu(k, "k")
        if v.get_device() != dev:
            _bad(f"v is on {v.device}, k on {k.device}")
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is not None:
                _vec(s, name, k.shape[2], torch.float32, dev)
                if k.dtype != torch.float8_e4m3fn:
                    _bad(f"{name} belongs to an 8-bit cache")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.gpu, self.dtype = k.device, dev, k.dtype
        self.pages, self.page, self.heads, self.dim = k.shape
        self.desc = _c.hts_kv_desc(self.pages, self.page, self.heads, self.dim, _c._dt(k.dtype), k.stride(0),
                                   k.stride(1), k.stride(2))
        # the descriptor's checks, once, before any step uses it
        _c.hts_paged_attn_workspace(0, self.heads, self.desc, 1)
        self._desc = ctypes.byref(self.desc)
        self._workspace = {}     # bytes by (requests, heads, width, window)

    def workspace_bytes(self, requests: int, q_heads: int, width: int, window: int = 0) -> int:
        """Bytes hts_paged_attn takes to split these sizes over their length."""
        key = (requests, q_heads, width, window)
        got = self._workspace.get(key)
        if got is None:
            got = _c.hts_paged_attn_workspace(requests, q_heads, self.desc, width, window)
            if len(self._workspace) > 1000:
                self._workspace.clear()
            self._workspace[key] = got
        return got


def kv_cache(pages: int, page: int, heads: int, dim: int, dtype, device="cuda", order: str = "token",
             k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None) -> KVCache:
    """A cache of zeros.  order "token": a page holds its tokens one after another, each with all heads;
    "head": a page holds its heads one after another, each with all the page's tokens."""
    if order not in ("token", "head"):
        _bad(f"order {order!r} is not token or head")
    shape = (pages, page, heads, dim) if order == "token" else (pages, heads, page, dim)

    def make():
        t = torch.zeros(shape, dtype=dtype, device=device)
        return t if order == "token" else t.transpose(1, 2)
    return KVCache(make(), make(), k_scale, v_scale)


@dataclasses.dataclass
class KVStep:
    """What a step writes: per request its length and first token, per token its slot and position."""
    lengths: torch.Tensor     # int32[B]
    starts: torch.Tensor      # int32[B + 1]
    slots: torch.Tensor       # int64[tokens], -1 where a token has no page
    positions: torch.Tensor   # int32[tokens], -1 past the step's last token
    head: torch.Tensor        # int32[1], first free-list entry the step has not taken

    @staticmethod
    def buffers(requests: int, tokens: int, device) -> "KVStep":
        """Buffers for a step, in one allocation."""
        sizes = (2 * tokens, tokens, requests, requests + 1, 1)
        slots, positions, lengths, starts, head = torch.empty(
            3 * tokens + 2 * requests + 2, dtype=torch.int32, device=device).split_with_sizes(sizes)
        return KVStep(lengths, starts, slots.view(torch.int64), positions, head)


def kv_step(cached: torch.Tensor, added: torch.Tensor, free_pages: torch.Tensor, block_table: torch.Tensor,
            page: int, tokens: int, free_head: Optional[torch.Tensor] = None, out: Optional[KVStep] = None,
            stream=None) -> KVStep:
    """Pages, slots and positions of one step that adds added[b] tokens to the cached[b] of request b.
    block_table (int32 [B, width], in place) gains the pages the new tokens open, taken from free_pages in
    order from entry free_head on.  ``tokens`` is the step's capacity: tokens past the batch's last one get
    slot and position -1.  Where head ends above free_pages.numel() the list was too short."""
    dev, B, i32 = _gpu(cached, "cached"), cached.numel(), torch.int32
    at_cached, at_added = _vec(cached, "cached", B, i32, dev), _vec(added, "added", B, i32, dev)
    n_free = free_pages.numel()
    at_free = _vec(free_pages, "free_pages", n_free, i32, dev)
    at_head = None if free_head is None else _vec(free_head, "free_head", 1, i32, dev)
    ldt = _table(block_table, B, dev)
    if tokens < 0:
        _bad(f"tokens={tokens} is negative", 3)
    if out is not None:
        for t, name, n in ((out.lengths, "lengths", B), (out.starts, "starts", B + 1),
                           (out.positions, "positions", tokens), (out.head, "head", 1)):
            _vec(t, name, n, i32, dev)
        _vec(out.slots, "slots", tokens, torch.int64, dev)
    with _scope(dev, stream):
        if out is None:
            out = KVStep.buffers(B, tokens, cached.device)
        _c._check(_c.lib().hts_kv_step(
            B, at_cached, at_added, page, at_free, n_free, at_head, block_table.data_ptr(), ldt, block_table.shape[1],
            tokens, out.lengths.data_ptr(), out.starts.data_ptr(), out.slots.data_ptr(), out.positions.data_ptr(),
            out.head.data_ptr(), _c._current_stream(dev)))
    return out


# --------------------------------------------------------------------------
# rotary positions
# --------------------------------------------------------------------------

@dataclasses.dataclass
class RopePlan:
    """Turns per position of each pair, on the device, with the layout they are used in."""
    turns: torch.Tensor       # float64[rot / 2]
    layout: int
    dim: int
    rot: int
    magnitude: float


def rope_plan(dim: int, rot: Optional[int] = None, theta: float = 10000.0, layout: str = "half",
              rule: str = "plain", factor: float = 1.0, context: float = 0.0, low: float = 1.0, high: float = 32.0,
              magnitude: float = 1.0, device="cuda") -> RopePlan:
    """The frequencies of rotary positions on the first ``rot`` entries of heads of ``dim`` (hts_rope_plan).
    layout "half" pairs entry i with i + rot/2, "interleaved" 2i with 2i + 1.  rule and factor stretch the
    positions past the trained context: "linear", "base" (a larger theta), "ramp" and "ramp_pairs" (only
    pairs with few turns over ``context``).  magnitude multiplies the rotated entries."""
    rot = dim if rot is None else rot
    lay, rul = _choice(_LAYOUTS, layout, "layout"), _choice(_RULES, rule, "rule")
    if rot > dim:
        _bad(f"rot={rot} exceeds the head size {dim}", 7)
    turns = _c.hts_rope_plan(_c.hts_rope_scaling(rot, rul, theta, factor, context, low, high))
    return RopePlan(torch.from_numpy(turns).to(device), lay, dim, rot, magnitude)


_rope_descs = {}


def _rope_desc(dtype, plan: RopePlan, q_heads: int, k_heads: int):
    key = (dtype, plan.layout, plan.dim, plan.rot, q_heads, k_heads, plan.magnitude)
    got = _rope_descs.get(key)
    if got is None:
        if len(_rope_descs) > 1000:
            _rope_descs.clear()
        d = _c.hts_rope_desc(_c._dt(dtype), plan.layout, plan.dim, plan.rot, q_heads, k_heads, plan.magnitude, 0)
        got = _rope_descs[key] = ctypes.byref(d)
    return got


def _rope_heads(x: torch.Tensor, name: str, dim: int) -> int:
    if x.dim() != 2 or x.shape[1] % dim:
        _bad(f"{name} must be [tokens, heads * {dim}]", 3)
    if x.dtype not in _16:
        _bad(f"{name} has type {x.dtype}, expected float16 or bfloat16", 2)
    return x.shape[1] // dim


def rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: torch.Tensor, plan: RopePlan,
         q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None):
    """Rotate q and k (either may be None) by their rows' positions (int32[T]), into q_out and k_out, or in
    place where none is given.  Rows with a negative position are left as they were.  Returns (q_out, k_out)."""
    ref = q if q is not None else k
    if ref is None:
        _bad("q and k are both missing")
    dev, T = _gpu(ref, "q" if ref is q else "k"), positions.numel()
    at = _vec(positions, "positions", T, torch.int32, dev)
    turns = _vec(plan.turns, "plan", plan.rot // 2, torch.float64, dev)
    q_out, k_out = q if q_out is None else q_out, k if k_out is None else k_out
    heads, args = [], []
    for x, out, name in ((q, q_out, "q"), (k, k_out, "k")):
        if x is None:
            heads.append(0)
            args += (None, 0, None, 0)
            continue
        heads.append(_rope_heads(x, name, plan.dim))
        n = x.shape[1]
        args += (x.data_ptr(), _lead(x, name, T, n, ref.dtype, dev),
                 out.data_ptr(), _lead(out, name + "_out", T, n, ref.dtype, dev))
    with _scope(dev, stream):
        _c._check(_c.lib().hts_rope(_rope_desc(ref.dtype, plan, *heads), turns, T, at, *args, _c._current_stream(dev)))
    return q_out, k_out


def rope_cache(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
               plan: RopePlan, cache: KVCache, q_out: Optional[torch.Tensor] = None, stream=None,
               starts: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotate q (into q_out, or in place) and write the rotated k, and v, of token t to slot slots[t] (int64)
    of the cache.  Tokens with a negative position are skipped; tokens with a slot outside the cache are not
    cached.  Slots must differ from one another.  Returns q_out.

    With ``starts`` (int32[B + 1], a step's) row b of q, k and v is request b's in place of token b's, for steps that
    add at most one token to a request: a request's row takes the position and slot of its token, starts[b]; one that
    adds none is skipped.  One that adds more, or whose token is past the step's capacity, gets NaN in q, and nothing of
    it is cached."""
    dev, tokens, dt, dim = _gpu(q, "q"), positions.numel(), q.dtype, plan.dim
    entry, T, rows = _c.lib().hts_rope_cache, tokens, ()
    if starts is not None:
        T = starts.numel() - 1
        if T < 0:
            _bad("starts must have an entry for each request, and one more", 3)
        entry, rows = _c.lib().hts_rope_cache_rows, (_vec(starts, "starts", T + 1, torch.int32, dev), tokens)
    if cache.gpu != dev:
        _bad(f"the cache is on GPU {cache.gpu}, q on GPU {dev}")
    hq, hk = _rope_heads(q, "q", dim), _rope_heads(k, "k", dim)
    nq, nk = hq * dim, hk * dim
    q_out = q if q_out is None else q_out
    ks, vs = cache.k_scale, cache.v_scale
    args = (_rope_desc(dt, plan, hq, hk), _vec(plan.turns, "plan", plan.rot // 2, torch.float64, dev), T, *rows,
            _vec(positions, "positions", tokens, torch.int32, dev), _vec(slots, "slots", tokens, torch.int64, dev),
            q.data_ptr(), _lead(q, "q", T, nq, dt, dev), q_out.data_ptr(), _lead(q_out, "q_out", T, nq, dt, dev),
            k.data_ptr(), _lead(k, "k", T, nk, dt, dev), v.data_ptr(), _lead(v, "v", T, nk, dt, dev), cache._desc,
            cache.k.data_ptr(), cache.v.data_ptr(), None if ks is None else ks.data_ptr(),
            None if vs is None else vs.data_ptr())
    with _scope(dev, stream):
        _c._check(entry(*args, _c._current_stream(dev)))
    return q_out


# --------------------------------------------------------------------------
# attention over the cache
# --------------------------------------------------------------------------

def paged_attn(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, lengths: torch.Tensor,
               scale: Optional[float] = None, window: int = 0, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """Attention of q [B, q heads * head size], one token per request, over the lengths[b] tokens of request
    b in the cache (its pages in block_table, int32 [B, width]), or over the last ``window`` of them.
    scale: default 1 / sqrt(head size).  lse (float32 [B, q heads]) receives the logarithm of the softmax's
    sum.  A request without tokens gets zeros.  The workspace is allocated here when none is given."""
    dev, dt = _gpu(q, "q"), q.dtype
    if cache.gpu != dev:
        _bad(f"the cache is on GPU {cache.gpu}, q on GPU {dev}")
    if q.dim() != 2 or not q.shape[1] or q.shape[1] % (cache.dim * cache.heads):
        _bad(f"q must be [requests, heads * {cache.dim}], its heads a multiple of the cache's {cache.heads}", 3)
    if dt not in _16:
        _bad(f"q has type {dt}, expected float16 or bfloat16", 2)
    B, n = q.shape
    heads = n // cache.dim
    ldq, ldt = _lead(q, "q", B, n, dt, dev), _table(block_table, B, dev)
    width, at_lengths = block_table.shape[1], _vec(lengths, "lengths", B, torch.int32, dev)
    ldo = n if out is None else _lead(out, "out", B, n, dt, dev)
    if lse is not None:
        _lead(lse, "lse", B, heads, torch.float32, dev)
        if not lse.is_contiguous():
            _bad("lse must be contiguous", 3)
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        _bad(f"workspace must be contiguous, on GPU {dev}", 3)
    ks, vs = cache.k_scale, cache.v_scale
    with _scope(dev, stream):
        if out is None:
            out = q.new_empty((B, n))
        if workspace is None:
            nbytes = cache.workspace_bytes(B, heads, width, window)
            if nbytes:
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        _c._check(_c.lib().hts_paged_attn(
            _c._DT[dt], B, heads, cache._desc, q.data_ptr(), ldq, cache.k.data_ptr(), cache.v.data_ptr(),
            None if ks is None else ks.data_ptr(), None if vs is None else vs.data_ptr(), block_table.data_ptr(), ldt,
            width, at_lengths, cache.dim ** -0.5 if scale is None else scale, window, out.data_ptr(), ldo,
            None if lse is None else lse.data_ptr(), None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.nbytes, _c._current_stream(dev)))
    return out


# --------------------------------------------------------------------------
# norms between blocks
# --------------------------------------------------------------------------

@dataclasses.dataclass
class Norm:
    """A norm over the row: kind "rms" or "layer", weight and bias [N] (none: ones, zeros)."""
    kind: str
    weight: Optional[torch.Tensor] = None
    bias: Optional[torch.Tensor] = None
    eps: float = 1e-6


_NO_NORM = Norm("none")
_norm_descs = {}


def residual_norm(block: Optional[torch.Tensor], residual: Optional[torch.Tensor], post: Optional[Norm] = None,
                  pre: Optional[Norm] = None, gate: Optional[torch.Tensor] = None, gate_act: str = "none",
                  scale: float = 1.0, residual_out: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, keep_residual: bool = True, out_dtype=None, stream=None):
    """The step between two blocks: r = residual + scale * act(gate) * post(block), y = pre(r), in one pass.

    block or residual may be None (zero).  gate: [N], one for all rows, or [M, N].  The residual stream has
    block's type or float32.  Returns (r, y): r rounded to the residual's type (into residual_out; None with
    keep_residual False), y in block's type (out_dtype where there is no block) from the unrounded r, into
    out; y is None where there is no pre norm.  residual_out may be residual, out may be block."""
    ref = block if block is not None else residual
    if ref is None or ref.dim() != 2:
        _bad("block or residual must be a [rows, width] matrix", 3)
    (M, N), dev = ref.shape, _gpu(ref, "block" if ref is block else "residual")
    post, pre = post or _NO_NORM, pre or _NO_NORM
    dt = block.dtype if block is not None else out.dtype if out is not None else out_dtype or residual.dtype
    if out_dtype is not None and out_dtype != dt:
        _bad(f"out_dtype {out_dtype}: y has the type of block and out, {dt}", 2)
    if dt not in _16:
        _bad(f"block and out of type {dt}: float16 or bfloat16 are taken", 2)
    rdt = residual.dtype if residual is not None else residual_out.dtype if residual_out is not None else dt
    if rdt is not dt and rdt is not torch.float32:
        _bad(f"the residual has type {rdt}, expected {dt} or float32", 2)
    key = (dt, rdt, post.kind, pre.kind, post.eps, pre.eps, scale, gate_act)
    desc = _norm_descs.get(key)
    if desc is None:
        if len(_norm_descs) > 1000:
            _norm_descs.clear()
        desc = _norm_descs[key] = ctypes.byref(_c.hts_norm_desc(
            _c._dt(dt), _c._dt(rdt), _choice(_NORMS, post.kind, "norm"), _choice(_NORMS, pre.kind, "norm"), post.eps,
            pre.eps, scale, _choice(_GATES, gate_act, "gate")))
    at_block = at_gate = at_r = None
    ldb = ldg = ldr = 0
    if block is not None:
        at_block, ldb = block.data_ptr(), _lead(block, "block", M, N, dt, dev)
    if gate is not None:
        at_gate = gate.data_ptr()
        if gate.dim() == 1:
            _vec(gate, "gate", N, dt, dev)
        else:
            ldg = _lead(gate, "gate", M, N, dt, dev)
    if residual is not None:
        at_r, ldr = residual.data_ptr(), _lead(residual, "residual", M, N, rdt, dev)
    w, what = post.weight, "a norm's weight or bias"
    post_w = None if w is None else _vec(w, what, N, dt, dev)
    w = post.bias
    post_b = None if w is None else _vec(w, what, N, dt, dev)
    w = pre.weight
    pre_w = None if w is None else _vec(w, what, N, dt, dev)
    w = pre.bias
    pre_b = None if w is None else _vec(w, what, N, dt, dev)
    with _scope(dev, stream):
        at_ro = at_y = None
        ldro = ldy = N
        if residual_out is not None:
            ldro = _lead(residual_out, "residual_out", M, N, rdt, dev)
        elif keep_residual:
            residual_out = torch.empty_like(ref) if ref.dtype is rdt and ref.is_contiguous() \
                else torch.empty((M, N), dtype=rdt, device=ref.device)
        if out is not None:
            ldy = _lead(out, "out", M, N, dt, dev)
        elif pre.kind != "none":
            out = torch.empty_like(ref) if ref.dtype is dt and ref.is_contiguous() \
                else torch.empty((M, N), dtype=dt, device=ref.device)
        if residual_out is not None:
            at_ro = residual_out.data_ptr()
        if out is not None:
            at_y = out.data_ptr()
        _c._check(_c.lib().hts_residual_norm(desc, M, N, at_block, ldb, post_w, post_b, at_gate, ldg, at_r, ldr, pre_w,
                                             pre_b, at_ro, ldro, at_y, ldy, _c._current_stream(dev)))
    return residual_out, out
