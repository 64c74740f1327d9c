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


def _here(device: torch.device, **tensors) -> None:
    """Every tensor given lives on this GPU."""
    if device.type != "cuda":
        _bad(f"tensors must be on a GPU, not on {device}")
    for name, t in tensors.items():
        if t is not None and t.device != device:
            _bad(f"{name} is on {t.device}, the other tensors on {device}")


def _matrix(t: torch.Tensor, name: str, rows: int, cols: int, dtypes) -> None:
    if t.dtype not in dtypes:
        _bad(f"{name} has type {t.dtype}, expected {' or '.join(map(str, dtypes))}", 2)
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        _bad(f"{name} has shape {tuple(t.shape)}, expected {(rows, cols)}", 3)
    if rows and cols > 1 and t.stride(1) != 1:
        _bad(f"the rows of {name} must be contiguous", 3)


def _vector(t: torch.Tensor, name: str, n: int, dtype) -> None:
    if t.dtype != dtype:
        _bad(f"{name} has type {t.dtype}, expected {dtype}", 2)
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        _bad(f"{name} must be a contiguous vector of {n} entries", 3)


@contextlib.contextmanager
def _switched(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            s = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=device)
            if s.device != device:
                _bad(f"the stream belongs to {s.device}, the tensors to {device}")
            with torch.cuda.stream(s):
                yield


def _scope(device: torch.device, stream):
    """Make the tensors' GPU and the call's stream current, for the launch and for what it allocates."""
    if stream is None and torch.cuda.current_device() == device.index:
        return contextlib.nullcontext()
    return _switched(device, stream)


def _rows(t: torch.Tensor) -> torch.Tensor:
    """The matrix with a leading dimension the library takes: a matrix of one row may carry any."""
    if t.dim() == 2 and t.shape[0] <= 1 and t.shape[1] and (t.stride(0) < t.shape[1] or t.stride(0) % 8):
        return t.as_strided(t.shape, ((t.shape[1] + 7) // 8 * 8, 1))
    return t


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
        _here(k.device, v=v, k_scale=k_scale, v_scale=v_scale)
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is not None:
                _vector(s, name, k.shape[2], torch.float32)
                if k.dtype != torch.float8_e4m3fn:
                    _bad(f"{name} belongs to an 8-bit cache")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.dtype = k.device, k.dtype
        self.pages, self.page, self.heads, self.dim = k.shape
        self.desc = _c.hts_kv_desc(self.pages, self.page, self.heads, self.dim, _c._dt(k.dtype), k.stride(0),
                                   k.stride(1), k.stride(2))
        # the descriptor's checks, once, before any step uses it
        _c.hts_paged_attn_workspace(0, self.heads, self.desc, 1)


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
        i32 = dict(dtype=torch.int32, device=device)
        return KVStep(torch.empty(requests, **i32), torch.empty(requests + 1, **i32),
                      torch.empty(tokens, dtype=torch.int64, device=device), torch.empty(tokens, **i32),
                      torch.empty(1, **i32))


def kv_step(cached: torch.Tensor, added: torch.Tensor, free_pages: torch.Tensor, block_table: torch.Tensor,
            page: int, tokens: int, free_head: Optional[torch.Tensor] = None, out: Optional[KVStep] = None,
            stream=None) -> KVStep:
    """Pages, slots and positions of one step that adds added[b] tokens to the cached[b] of request b.
    block_table (int32 [B, width], in place) gains the pages the new tokens open, taken from free_pages in
    order from entry free_head on.  ``tokens`` is the step's capacity: tokens past the batch's last one get
    slot and position -1.  Where head ends above free_pages.numel() the list was too short."""
    dev, B = cached.device, cached.numel()
    _here(dev, added=added, free_pages=free_pages, block_table=block_table, free_head=free_head)
    _vector(cached, "cached", B, torch.int32)
    _vector(added, "added", B, torch.int32)
    _vector(free_pages, "free_pages", free_pages.numel(), torch.int32)
    if block_table.dim() != 2:
        _bad("block_table must be [requests, pages of a request]", 3)
    _matrix(block_table, "block_table", B, block_table.shape[1], (torch.int32,))
    if tokens < 0:
        _bad(f"tokens={tokens} is negative", 3)
    if free_head is not None:
        _vector(free_head, "free_head", 1, torch.int32)
    with _scope(dev, stream):
        if out is None:
            out = KVStep.buffers(B, tokens, dev)
        else:
            _here(dev, lengths=out.lengths, starts=out.starts, slots=out.slots, positions=out.positions, head=out.head)
            _vector(out.lengths, "lengths", B, torch.int32)
            _vector(out.starts, "starts", B + 1, torch.int32)
            _vector(out.slots, "slots", tokens, torch.int64)
            _vector(out.positions, "positions", tokens, torch.int32)
            _vector(out.head, "head", 1, torch.int32)
        if B <= 1 and block_table.stride(0) < block_table.shape[1]:
            block_table = block_table.as_strided(block_table.shape, (block_table.shape[1], 1))
        _c.hts_kv_step(cached, added, page, free_pages, free_head, block_table, out.lengths, out.starts, out.slots,
                       out.positions, out.head)
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


def _rope_checks(q, k, positions, plan, q_out, k_out):
    ref = q if q is not None else k
    if ref is None:
        _bad("q and k are both missing")
    T, dev = positions.numel(), ref.device
    _here(dev, q=q, k=k, q_out=q_out, k_out=k_out, positions=positions, turns=plan.turns)
    _vector(positions, "positions", T, torch.int32)
    heads = []
    for x, out, name in ((q, q_out, "q"), (k, k_out, "k")):
        if x is None:
            heads.append(0)
            continue
        if x.dim() != 2 or x.shape[1] % plan.dim:
            _bad(f"{name} must be [tokens, heads * {plan.dim}]", 3)
        _matrix(x, name, T, x.shape[1], _16)
        if x.dtype != ref.dtype:
            _bad("q and k must share a type", 2)
        if out is not None:
            _matrix(out, name + "_out", T, x.shape[1], (x.dtype,))
        heads.append(x.shape[1] // plan.dim)
    return dev, heads, _c.hts_rope_desc(_c._dt(ref.dtype), plan.layout, plan.dim, plan.rot, heads[0], heads[1],
                                        plan.magnitude, 0)


def rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: torch.Tensor, plan: RopePlan,
         q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None):
    """Rotate q and k (either may be None) by their rows' positions (int32[T]), into q_out and k_out, or in
    place where none is given.  Rows with a negative position are left as they were.  Returns (q_out, k_out)."""
    dev, _, desc = _rope_checks(q, k, positions, plan, q_out, k_out)
    q_out, k_out = q if q_out is None else q_out, k if k_out is None else k_out
    with _scope(dev, stream):
        r = [None if x is None else _rows(x) for x in (q, q_out, k, k_out)]
        _c.hts_rope(desc, plan.turns, positions, *r)
    return q_out, k_out


def rope_cache(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
               plan: RopePlan, cache: KVCache, q_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rotate q (into q_out, or in place) and write the rotated k, and v, of token t to slot slots[t] (int64)
    of the cache.  Tokens with a negative position are skipped; tokens with a slot outside the cache are not
    cached.  Slots must differ from one another.  Returns q_out."""
    dev, heads, desc = _rope_checks(q, k, positions, plan, q_out, None)
    _here(dev, v=v, slots=slots, k_cache=cache.k)
    T = positions.numel()
    _matrix(v, "v", T, k.shape[1], (k.dtype,))
    _vector(slots, "slots", T, torch.int64)
    q_out = q if q_out is None else q_out
    with _scope(dev, stream):
        _c.hts_rope_cache(desc, plan.turns, positions, slots, _rows(q), _rows(q_out), _rows(k), _rows(v), cache.desc,
                          cache.k, cache.v, cache.k_scale, cache.v_scale)
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
    dev, B = q.device, q.shape[0]
    _here(dev, k_cache=cache.k, block_table=block_table, lengths=lengths, out=out, lse=lse, workspace=workspace)
    if q.dim() != 2 or not q.shape[1] or q.shape[1] % (cache.dim * cache.heads):
        _bad(f"q must be [requests, heads * {cache.dim}], its heads a multiple of the cache's {cache.heads}", 3)
    _matrix(q, "q", B, q.shape[1], _16)
    heads = q.shape[1] // cache.dim
    if block_table.dim() != 2:
        _bad("block_table must be [requests, pages of a request]", 3)
    _matrix(block_table, "block_table", B, block_table.shape[1], (torch.int32,))
    _vector(lengths, "lengths", B, torch.int32)
    if out is not None:
        _matrix(out, "out", B, q.shape[1], (q.dtype,))
    if lse is not None:
        _matrix(lse, "lse", B, heads, (torch.float32,))
        if not lse.is_contiguous():
            _bad("lse must be contiguous", 3)
    with _scope(dev, stream):
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        if workspace is None:
            nbytes = _c.hts_paged_attn_workspace(B, heads, cache.desc, block_table.shape[1], window)
            if nbytes:
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        elif not workspace.is_contiguous():
            _bad("workspace must be contiguous", 3)
        if B <= 1 and block_table.stride(0) < block_table.shape[1]:
            block_table = block_table.as_strided(block_table.shape, (block_table.shape[1], 1))
        _c.hts_paged_attn(heads, cache.desc, _rows(q), cache.k, cache.v, block_table, lengths,
                          cache.dim ** -0.5 if scale is None else scale, _rows(out), cache.k_scale, cache.v_scale,
                          window, lse, workspace)
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
    (M, N), dev = ref.shape, ref.device
    post, pre = post or _NO_NORM, pre or _NO_NORM
    kinds = _choice(_NORMS, post.kind, "norm"), _choice(_NORMS, pre.kind, "norm")
    act = _choice(_GATES, gate_act, "gate")
    _here(dev, block=block, residual=residual, gate=gate, residual_out=residual_out, out=out, post_weight=post.weight,
          post_bias=post.bias, pre_weight=pre.weight, pre_bias=pre.bias)
    dt = block.dtype if block is not None else out.dtype if out is not None else out_dtype or residual.dtype
    if dt not in _16:
        _bad(f"block and out of type {dt}: float16 or bfloat16 are taken", 2)
    rdt = residual.dtype if residual is not None else residual_out.dtype if residual_out is not None else dt
    if block is not None:
        _matrix(block, "block", M, N, (dt,))
    if residual is not None:
        _matrix(residual, "residual", M, N, (dt, torch.float32))
    if residual_out is not None:
        _matrix(residual_out, "residual_out", M, N, (rdt,))
    if out is not None:
        _matrix(out, "out", M, N, (dt,))
    if gate is not None:
        if gate.dim() == 1:
            _vector(gate, "gate", N, dt)
        else:
            _matrix(gate, "gate", M, N, (dt,))
    for n, name in ((post, "post"), (pre, "pre")):
        for t, what in ((n.weight, "weight"), (n.bias, "bias")):
            if t is not None:
                _vector(t, f"{name}_{what}", N, dt)
    desc = _c.hts_norm_desc(_c._dt(dt), _c._dt(rdt), kinds[0], kinds[1], post.eps, pre.eps, scale, act)
    with _scope(dev, stream):
        if residual_out is None and keep_residual:
            residual_out = torch.empty((M, N), dtype=rdt, device=dev)
        if out is None and kinds[1]:
            out = torch.empty((M, N), dtype=dt, device=dev)
        r = [None if t is None else _rows(t) for t in (block, gate, residual, residual_out, out)]
        _c.hts_residual_norm(desc, M, N, r[0], post.weight, post.bias, r[1], r[2], pre.weight, pre.bias, r[3], r[4])
    return residual_out, out
