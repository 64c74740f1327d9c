"""Tensor-level helpers of the 8-bit linear layers: E4M3 values with a scale for each block of 128.

    w = ScaledWeight(values, scale)                 an 8-bit checkpoint's weight, or ScaledWeight.quantize(w16)
    q, scale = quantize_rows(x)                     activations: a scale for each row and 128 columns
    y = scaled_gemm(q, scale, w)                    the product
    h = scaled_gated(q, scale, gate, up)            act(x gate^T) * (x up^T); out_dtype=float8_e4m3fn: (h, scale)
    y = scaled_mlp(x, gate, up, down)               a decoder block's feed-forward part on 16-bit rows

As in the rest of the package these only check and marshal arguments; the work is in the HIP kernels.  All tensors of a
call live on one GPU; the call runs on ``stream`` (default: that GPU's current stream), and what it allocates belongs to
that stream.  Every call can be captured in a HIP graph (give ``out`` and ``workspace`` there, or keep what is returned at
capture).  The scales of rows are [rows, blocks] tensors whose rows are consecutive (stride 1): one block's scales lie
together, as the kernels read them.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

import tile_gemm_amd as _c
from .serving import _16, _bad, _choice, _explain, _gpu, _lead, _scope

_ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
_E4M3 = torch.float8_e4m3fn
_OUT = (torch.bfloat16, torch.float16, torch.float32)
_CODE = {t: _c._dt(t) for t in _OUT + (_E4M3,)}


def _blocks(n: int) -> int:
    return -(-n // 128)


def _row_scale(t: torch.Tensor, name: str, rows: int, cols: int, dev: int) -> int:
    """Leading dimension (between blocks) of the scales of rows."""
    if t.dtype is not torch.float32 or t.get_device() != dev or tuple(t.shape) != (rows, _blocks(cols)):
        _explain(t, name, rows, _blocks(cols), (torch.float32,), dev)
    if rows > 1 and t.stride(0) != 1:
        _bad(f"{name} must have consecutive rows (stride 1 in its first axis): x_scale.t().contiguous().t()", 3)
    return t.stride(1) if t.shape[1] > 1 else max(rows, 1)


def _new_scale(rows: int, cols: int, device) -> torch.Tensor:
    return torch.empty_strided((rows, _blocks(cols)), (1, rows), dtype=torch.float32, device=device)


class ScaledWeight:
    """A weight [N, K] in 8 bits: float8_e4m3fn values (rows any multiple of 16 bytes apart) and a float32 scale
    [ceil(N / 128), ceil(K / 128)] for each block of 128 rows and columns.  Stands for values * scale."""

    def __init__(self, values: torch.Tensor, scale: torch.Tensor):
        if values.dim() != 2 or not values.shape[0] or not values.shape[1]:
            _bad("values must be a [rows, columns] matrix", 3)
        dev = _gpu(values, "values")
        self.N, self.K = values.shape
        ld = _lead(values, "values", self.N, self.K, _E4M3, dev) if self.N > 1 else (self.K + 15) // 16 * 16
        if values.dtype != _E4M3:
            _bad(f"values have type {values.dtype}, expected {_E4M3}", 2)
        if self.N == 1 and self.K > 1 and values.stride(1) != 1:
            _bad("values must be contiguous along their rows", 3)
        lds = _lead(scale, "scale", _blocks(self.N), _blocks(self.K), torch.float32, dev)
        if lds < _blocks(self.K):
            _bad(f"scale's rows are {lds} apart and {_blocks(self.K)} long (an expanded scale: scale.contiguous())", 3)
        self.values, self.scale, self.device, self.gpu = values, scale, values.device, dev
        self.desc = _c.hts_scaled_weight(values.data_ptr(), ld, scale.data_ptr(), lds)
        self._desc = ctypes.byref(self.desc)
        self._workspace = {}     # bytes by (rows, what)
        # the shape's checks, once, before any product uses it
        _c.hts_scaled_gemm_workspace(0, self.N, self.K)

    @property
    def shape(self):
        return (self.N, self.K)

    @property
    def dtype(self):
        return _E4M3

    @staticmethod
    def quantize(w: torch.Tensor, stream=None) -> "ScaledWeight":
        """A 16-bit or float32 weight [N, K] in 8 bits, each block scaled to E4M3's range."""
        dev = _gpu(w, "w")
        if w.dim() != 2:
            _bad("w must be a [rows, columns] matrix", 3)
        N, K = w.shape
        ldw = _lead(w, "w", N, K, w.dtype, dev)
        with _scope(dev, stream):
            values = torch.empty((N, K), dtype=_E4M3, device=w.device)
            scale = torch.empty((_blocks(N), _blocks(K)), dtype=torch.float32, device=w.device)
            _c._check(_c.lib().hts_quantize_weight(_c._dt(w.dtype), N, K, w.data_ptr(), ldw, values.data_ptr(), K,
                                                   scale.data_ptr(), _blocks(K), _c._current_stream(dev)))
            return ScaledWeight(values, scale)

    def _bytes(self, key, ask) -> int:
        got = self._workspace.get(key)
        if got is None:
            if len(self._workspace) > 1000:
                self._workspace.clear()
            got = self._workspace[key] = ask()
        return got


def quantize_rows(x: torch.Tensor, out: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                  stream=None):
    """x [M, K] (16-bit or float32) to E4M3 values and their scales: a / 448 for the largest magnitude a of each row
    and 128 columns.  Returns (values [M, K], scale [M, ceil(K / 128)], its rows consecutive)."""
    dev = _gpu(x, "x")
    if x.dim() != 2:
        _bad("x must be a [rows, columns] matrix", 3)
    M, K = x.shape
    if x.dtype not in _OUT:
        _bad(f"x has type {x.dtype}, expected float16, bfloat16 or float32", 2)
    ldx = _lead(x, "x", M, K, x.dtype, dev)
    ldq = K if out is None else _lead8(out, "out", M, K, dev)
    lds = M if scale is None else _row_scale(scale, "scale", M, K, dev)
    with _scope(dev, stream):
        if out is None:
            out = torch.empty((M, K), dtype=_E4M3, device=x.device)
        if scale is None:
            scale = _new_scale(M, K, x.device)
        _c._check(_c.lib().hts_quantize_rows(_CODE[x.dtype], M, K, x.data_ptr(), ldx, out.data_ptr(), ldq,
                                             scale.data_ptr(), lds, _c._current_stream(dev)))
    return out, scale


def _lead8(t: torch.Tensor, name: str, rows: int, cols: int, dev: int) -> int:
    ld = _lead(t, name, rows, cols, _E4M3, dev)
    return ld if rows > 1 else (cols + 15) // 16 * 16


def _rows(x: torch.Tensor, x_scale: torch.Tensor, w: ScaledWeight):
    """Checked (rows, leading dimensions of x and its scales) of a product's input."""
    dev = w.gpu
    if x.dim() != 2:
        _bad("x must be a [rows, columns] matrix", 3)
    M = x.shape[0]
    return M, _lead8(x, "x", M, w.K, dev), _row_scale(x_scale, "x_scale", M, w.K, dev)


def _out(out, out_dtype, M: int, N: int, dtypes, dev: int, device):
    """Checked (out, leading dimension, type)."""
    if out is None:
        if out_dtype not in dtypes:
            _bad(f"out_dtype {out_dtype} is not one of {', '.join(map(str, dtypes))}", 2)
        ld = (N + 3) // 4 * 4
        return None, ld, out_dtype
    if out.dtype not in dtypes:
        _bad(f"out has type {out.dtype}, expected {' or '.join(map(str, dtypes))}", 2)
    ld = _lead(out, "out", M, N, out.dtype, dev)
    return out, ld if M > 1 else (N + 15) // 16 * 16, out.dtype


def _new_out(M: int, N: int, ld: int, dtype, device) -> torch.Tensor:
    out = torch.empty((M, ld), dtype=dtype, device=device)
    return out if ld == N else out[:, :N]


def _space(workspace: Optional[torch.Tensor], nbytes: int, dev: int, device):
    """(tensor kept alive, address, bytes) of a call's workspace, allocated here where none is given."""
    if workspace is None:
        if not nbytes:
            return None, None, 0
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _bad(f"workspace must be contiguous, on GPU {dev}", 3)
    return workspace, workspace.data_ptr(), workspace.nbytes


def scaled_gemm(x: torch.Tensor, x_scale: torch.Tensor, w: ScaledWeight, out_dtype=torch.bfloat16,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """y [M, N] = (x * x_scale) (w)^T from 8-bit values, block by block of K, summed in 32 bits and rounded once to
    bfloat16, float16 or float32.  16-bit outputs come from 8-bit matrix instructions (1.5e-5 of the 2-norm, below their
    rounding); float32 ones lose no products, at up to twice the time.  The workspace of a split product is allocated
    here when none is given."""
    M, ldx, lds = _rows(x, x_scale, w)
    dev, N = w.gpu, w.N
    out, ldy, dt = _out(out, out_dtype, M, N, _OUT, dev, w.device)
    with _scope(dev, stream):
        if out is None:
            out = _new_out(M, N, ldy, dt, w.device)
        keep, at, nbytes = _space(workspace, w._bytes((M,), lambda: _c.hts_scaled_gemm_workspace(M, N, w.K)), dev, w.device)
        _c._check(_c.lib().hts_scaled_gemm(M, N, w.K, x.data_ptr(), ldx, x_scale.data_ptr(), lds, w._desc, out.data_ptr(),
                                           ldy, _CODE[dt], at, nbytes, _c._current_stream(dev)))
    return out


def scaled_gated(x: torch.Tensor, x_scale: torch.Tensor, gate: ScaledWeight, up: ScaledWeight, act: str = "silu",
                 out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None, out_scale: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """h [M, N] = act(x gate^T) * (x up^T), both products and the step between them in one pass.  act: "silu", "gelu" or
    "gelu_tanh".  With out_dtype float8_e4m3fn returns (h, scale), quantised as quantize_rows does from the unrounded
    sums: the input of the next product."""
    M, ldx, lds = _rows(x, x_scale, gate)
    code = _choice(_ACTS, act, "act")
    dev, N, K = gate.gpu, gate.N, gate.K
    if up.shape != gate.shape or up.gpu != dev:
        _bad(f"up is {up.N} x {up.K} on {up.device}, gate {N} x {K} on {gate.device}", 3)
    out, ldh, dt = _out(out, out_dtype, M, N, _OUT + (_E4M3,), dev, gate.device)
    at_scale, ldhs = None, 0
    if dt is _E4M3:
        ldhs = M if out_scale is None else _row_scale(out_scale, "out_scale", M, N, dev)
    elif out_scale is not None:
        _bad("out_scale belongs to a float8_e4m3fn output")
    with _scope(dev, stream):
        if out is None:
            out = _new_out(M, N, ldh, dt, gate.device)
        if dt is _E4M3:
            if out_scale is None:
                out_scale = _new_scale(M, N, gate.device)
            at_scale = out_scale.data_ptr()
        keep, at, nbytes = _space(
            workspace, gate._bytes((M, dt), lambda: _c.hts_scaled_gated_workspace(M, N, K, dt)), dev, gate.device)
        _c._check(_c.lib().hts_scaled_gated(code, M, N, K, x.data_ptr(), ldx, x_scale.data_ptr(), lds, gate._desc, up._desc,
                                            out.data_ptr(), ldh, _CODE[dt], at_scale, ldhs, at, nbytes,
                                            _c._current_stream(dev)))
    return out if out_scale is None else (out, out_scale)


def scaled_mlp(x: torch.Tensor, gate: ScaledWeight, up: ScaledWeight, down: ScaledWeight, act: str = "silu",
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """A decoder block's feed-forward part: 16-bit rows x [M, hidden] quantised, act(x gate^T) * (x up^T) quantised, and
    the down projection, in x's type.  out may be x."""
    dev, hidden, inner = gate.gpu, gate.K, gate.N
    if x.dim() != 2:
        _bad("x must be a [rows, columns] matrix", 3)
    if x.dtype not in _16:
        _bad(f"x has type {x.dtype}, expected float16 or bfloat16", 2)
    M = x.shape[0]
    ldx = _lead(x, "x", M, hidden, x.dtype, dev)
    code = _choice(_ACTS, act, "act")
    for name, w, shape in (("up", up, (inner, hidden)), ("down", down, (hidden, inner))):
        if w.shape != shape or w.gpu != dev:
            _bad(f"{name} is {w.N} x {w.K} on {w.device}, expected {shape[0]} x {shape[1]} on {gate.device}", 3)
    ldy = hidden if out is None else _lead(out, "out", M, hidden, x.dtype, dev)
    with _scope(dev, stream):
        if out is None:
            out = torch.empty((M, hidden), dtype=x.dtype, device=x.device)
        keep, at, nbytes = _space(
            workspace, gate._bytes((M, "mlp"), lambda: _c.hts_scaled_mlp_workspace(M, hidden, inner)), dev, x.device)
        _c._check(_c.lib().hts_scaled_mlp(code, _CODE[x.dtype], M, hidden, inner, x.data_ptr(), ldx, gate._desc, up._desc,
                                          down._desc, out.data_ptr(), ldy, at, nbytes, _c._current_stream(dev)))
    return out
