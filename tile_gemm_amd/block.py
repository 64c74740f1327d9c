"""The linear layers of a LLaMA-style decoder block on hybrid tile-sparse weights.

The pages prune the linear layers of LLaMA-family models and report speed at the level of the
whole model ("PATCH: Learnable Tile-level Hybrid Sparsity for LLMs", section 4, speed).  The
closest weight-free analogue this library can run is one decoder block's seven projections
back to back:

    q = X Wq^T,  k = X Wk^T,  v = X Wv^T,  o = A Wo^T,
    gate = X Wg^T,  up = X Wu^T,  h = silu(gate) * up,  down = h Wd^T

with every W either a packed hybrid weight (hts_gemm), a row-major dense one
(hts_dense_gemm, the same-library baseline) or a dense 8-bit one with a scale for each block of 128
(ScaledWeight: the projections of one input share its hts_quantize_rows and go through hts_scaled_gemm; 8-bit
gate and up through hts_scaled_gated, and with an 8-bit down through hts_scaled_mlp).  In ``forward`` the output projection
reads A = q in place of the attention output, which keeps the shapes and the data dependence of the block.
Every call is enqueued on the current stream, so the whole step can be captured in one HIP
graph.

``decode`` runs the whole block for one new token per request, on the steps around the products
(``serving``): norm, q / k / v, rotary positions with k and v written to a paged cache, attention
over the cache, o, and the residual additions with the norms around them.  A step of a model is
one ``kv_step`` for all layers, then ``decode`` per layer:

    step = kv_step(cached, ones, free_pages, table, cache.page, B, free_head=head)
    x, r = embed(tokens), None
    for layer in layers:
        x, r = decode(x, r, layer, step, table, plan)
    cached, head = step.lengths, step.head
"""
from __future__ import annotations

import dataclasses
import math
from typing import Dict, Optional

import torch

from . import (HTSError, KVCache, KVStep, Norm, PackedWeight, RopePlan, ScaledWeight, dense_gemm, gemm, gemm_silu_mul,
               paged_attn, quantize_rows, residual_norm, rope_cache, scaled_gated, scaled_gemm, scaled_mlp, silu_mul)

PROJECTIONS = ("q", "k", "v", "o", "gate", "up", "down")


def buffers(M: int, weights: Dict[str, object], dtype, device) -> Dict[str, torch.Tensor]:
    """Output buffers of every step for M tokens."""
    def rows(w):
        return w.N if isinstance(w, PackedWeight) else w.shape[0]
    out = {name: torch.empty((M, rows(weights[name])), dtype=dtype, device=device) for name in PROJECTIONS}
    out["h"] = torch.empty_like(out["gate"])
    return out


def _linear(x: torch.Tensor, w, out: torch.Tensor) -> torch.Tensor:
    if isinstance(w, PackedWeight):
        return gemm(x, w, out=out)
    if isinstance(w, ScaledWeight):
        return scaled_gemm(*quantize_rows(x), w, out=out)
    return dense_gemm(x, w, out=out)


def _linears(x: torch.Tensor, names, weights: Dict[str, object], bufs: Dict[str, torch.Tensor]) -> None:
    """Several projections of one input, quantised once for those in 8 bits."""
    scaled = [n for n in names if isinstance(weights[n], ScaledWeight)]
    if scaled:
        q, scale = quantize_rows(x)
        for n in scaled:
            scaled_gemm(q, scale, weights[n], out=bufs[n])
    for n in names:
        if n not in scaled:
            _linear(x, weights[n], bufs[n])


def _mlp(x: torch.Tensor, w: Dict[str, object], bufs: Dict[str, torch.Tensor]) -> torch.Tensor:
    """down(silu(gate x) * (up x)) in the fewest steps that the weights allow."""
    scaled = [isinstance(w[n], ScaledWeight) for n in ("gate", "up", "down")]
    if all(scaled):
        return scaled_mlp(x, w["gate"], w["up"], w["down"], out=bufs["down"])
    if scaled[0] and scaled[1]:
        scaled_gated(*quantize_rows(x), w["gate"], w["up"], out=bufs["h"])
    elif isinstance(w["up"], PackedWeight):
        _linear(x, w["gate"], bufs["gate"])
        gemm_silu_mul(x, w["up"], bufs["gate"], out=bufs["h"])
    else:
        _linears(x, ("gate", "up"), w, bufs)
        silu_mul(bufs["gate"], bufs["up"], out=bufs["h"])
    return _linear(bufs["h"], w["down"], bufs["down"])


def forward(X: torch.Tensor, weights: Dict[str, object], bufs: Dict[str, torch.Tensor],
            fused: bool = False) -> torch.Tensor:
    """One block step on M = X.shape[0] tokens; returns the down-projection output.  fused (packed
    up weight only): the up product writes silu(gate) * up itself (hts_gemm_silu_mul) instead of
    writing up for a separate elementwise pass.  8-bit gate and up weights take the steps that ``decode`` takes
    (the buffers of steps inside a call are then not written)."""
    fuse = fused and isinstance(weights["up"], PackedWeight)
    scaled = isinstance(weights["gate"], ScaledWeight) and isinstance(weights["up"], ScaledWeight)
    _linears(X, ("q", "k", "v") + (() if scaled else ("gate",)) + (() if scaled or fuse else ("up",)), weights, bufs)
    _linear(bufs["q"], weights["o"], bufs["o"])          # attention output stand-in: A = q
    if scaled:
        return _mlp(X, weights, bufs)
    if fuse:
        gemm_silu_mul(X, weights["up"], bufs["gate"], out=bufs["h"])
    else:
        silu_mul(bufs["gate"], bufs["up"], out=bufs["h"])
    return _linear(bufs["h"], weights["down"], bufs["down"])


def kept_flops(M: int, weights: Dict[str, object]) -> float:
    """Algorithmic flops of one step: 2 M (kept weights) over the seven projections."""
    total = 0
    for name in PROJECTIONS:
        w = weights[name]
        if isinstance(w, PackedWeight):
            total += w.N * w.K - w.sizes["n_sparse"] * w.desc.bn * w.desc.bk // 2
        else:
            total += w.shape[0] * w.shape[1]
    return 2.0 * M * total


@dataclasses.dataclass
class Layer:
    """A decoder block: its seven projections (packed, row-major or in 8 bits with scales), its norms and its cache.

    input_norm and mlp_norm come before attention and the MLP; the optional post norms, gates ([hidden], or one
    for each token) and residual_scale apply to what the two write back to the residual stream:
    x + residual_scale * gate * post(block(norm(x)))."""
    weights: Dict[str, object]
    cache: KVCache
    input_norm: Norm
    mlp_norm: Norm
    post_attn_norm: Optional[Norm] = None
    post_mlp_norm: Optional[Norm] = None
    attn_gate: Optional[torch.Tensor] = None
    mlp_gate: Optional[torch.Tensor] = None
    residual_scale: float = 1.0
    window: int = 0
    attn_scale: Optional[float] = None       # default: 1 / sqrt(head size)

    def __post_init__(self):
        # The products take any input that their leading dimension lets through: the block's own shapes are held here.
        # 8-bit weights with scales take rows of either 16-bit type.
        shape = {n: ((w.N, w.K) if isinstance(w, PackedWeight) else tuple(w.shape), w.dtype)
                 for n, w in self.weights.items()}
        if sorted(shape) != sorted(PROJECTIONS):
            raise HTSError(1, f"a block has the projections {', '.join(PROJECTIONS)}")
        (nq, hidden), _ = shape["q"]
        self.hidden = hidden
        plain = [n for n in PROJECTIONS if not isinstance(self.weights[n], ScaledWeight)]
        self.dtype = dt = shape[plain[0]][1] if plain else None      # None: the rows' own
        nk, inner = self.cache.heads * self.cache.dim, shape["gate"][0][0]
        want = dict(q=(nq, hidden), k=(nk, hidden), v=(nk, hidden), o=(hidden, nq), gate=(inner, hidden),
                    up=(inner, hidden), down=(hidden, inner))
        for n, (got, t) in shape.items():
            if n in plain and (t != dt or t not in (torch.float16, torch.bfloat16)):
                raise HTSError(2, f"{n} has type {t}: a block's weights share one 16-bit type")
            if got != want[n]:
                raise HTSError(3, f"{n} is {got[0]} x {got[1]}, the block's other shapes ask for {want[n][0]} x {want[n][1]}")
        # what attention would refuse after the step's keys and values are in the cache
        if nq % nk:
            raise HTSError(3, f"q has {nq} rows, not a multiple of the cache's {self.cache.heads} heads of {self.cache.dim}")
        if self.window < 0:
            raise HTSError(3, f"window={self.window} is negative")
        if self.attn_scale is not None and not math.isfinite(self.attn_scale):
            raise HTSError(1, "attn_scale is not finite")


def decode(x: torch.Tensor, residual: Optional[torch.Tensor], layer: Layer, step: KVStep, block_table: torch.Tensor,
           plan: RopePlan, bufs: Optional[Dict[str, torch.Tensor]] = None):
    """One block on one new token per request: row b of x [B, hidden] is request b's, the output of the block before
    (its MLP, not yet added) with that block's residual stream, or the embedding with residual None.  Returns (x, residual) for
    the next block: the MLP's output and the stream it is to be added to.  The layer's post_mlp_norm, gate
    and scale are applied here, so that the next block only adds: give the last block's pair to
    residual_norm(x, residual, pre=final_norm).

    step and block_table come from kv_step with B tokens of capacity and at most one token added to a request.  The row
    of a request that adds none (padding, paused or finished, wherever it stands) is carried along and changes no
    cache entry; what comes out in it means nothing.  A request that adds more than one gets NaN in its row."""
    w, B = layer.weights, x.shape[0]
    if x.dim() != 2 or x.shape[1] != layer.hidden:
        raise HTSError(3, f"x has shape {tuple(x.shape)}, the block's hidden size is {layer.hidden}")
    if layer.dtype is not None and x.dtype != layer.dtype:
        raise HTSError(2, f"x has type {x.dtype}, the block's weights {layer.dtype}")
    if step.positions.numel() != B or step.lengths.numel() != B or step.starts.numel() != B + 1:
        raise HTSError(3, f"x has {B} rows, the step {step.lengths.numel()} requests and {step.positions.numel()} tokens")
    if bufs is None:
        bufs = buffers(B, w, x.dtype, x.device)
    # r = residual + x, y = norm(r)
    r, y = residual_norm(x, residual, pre=layer.input_norm)
    _linears(y, ("q", "k", "v"), w, bufs)
    rope_cache(bufs["q"], bufs["k"], bufs["v"], step.positions, step.slots, plan, layer.cache, starts=step.starts)
    a = paged_attn(bufs["q"], layer.cache, block_table, step.lengths, layer.attn_scale, layer.window)
    _linear(a, w["o"], bufs["o"])
    r, y = residual_norm(bufs["o"], r, post=layer.post_attn_norm, pre=layer.mlp_norm, gate=layer.attn_gate,
                         scale=layer.residual_scale, residual_out=r)
    out = _mlp(y, w, bufs)
    if layer.post_mlp_norm is not None or layer.mlp_gate is not None or layer.residual_scale != 1.0:
        out, _ = residual_norm(out, None, post=layer.post_mlp_norm, gate=layer.mlp_gate, scale=layer.residual_scale)
    return out, r
