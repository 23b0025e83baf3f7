"""Torch-facing wrappers of the entry points around the layers: the norm between two blocks,
rows in 8 bits and their product, and the choice of the next token.

As in serve.py: each wrapper checks dtypes, devices and shapes, allocates outputs and workspaces
with torch on the inputs' device, and calls libawq on torch's current stream of that device; all
arithmetic happens in the library's HIP kernels.  A decoding step makes these calls on little
data, so the wrappers are kept short.

As everywhere in the library every tensor starts on 16 bytes, the small ones too: a slice such as
u[i] of fp32 [steps][5] does not, and is refused by name; its clone does.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Union

import torch

from ._lib import check, load
from .api import _need
from .serve import _like, _raw_stream, _scratch

NORM_KINDS = ("rms", "layer")

_F16, _F32, _I32, _I8 = torch.float16, torch.float32, torch.int32, torch.int8
_FLOATS = (_F16, _F32)

_current_device = torch._C._cuda_getDevice  # of the calling thread


def _run(index: int, fn, *args) -> None:
    """fn(*args, stream) with the device current and its current stream; raises on a status."""
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        check(status)


def _matrix(t: torch.Tensor, name: str, dtypes, index: int):
    """(rows, columns, elements from one row to the next) of a matrix of one of the dtypes on the given device
    (-1: any GPU) whose rows are contiguous; any stride between rows (a single row has no next)."""
    if isinstance(t, torch.Tensor) and t.dim() == 2 and t.dtype in dtypes:
        device = t.get_device()
        if device >= 0 and (device == index or index < 0):
            T, N = t.shape
            if t.is_contiguous():
                return T, N, N
            row, column = t.stride()
            if column == 1 or N == 1:
                return T, N, row if T > 1 else N
            raise ValueError(f"{name} must be contiguous within each row")
    if isinstance(t, torch.Tensor) and t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    _need(t, name, dtypes[0] if not isinstance(t, torch.Tensor) else t.dtype, 2)
    raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _vector(t: torch.Tensor, name: str, dtype: torch.dtype, n: int, index: int) -> int:
    """The pointer of a vector of n."""
    if isinstance(t, torch.Tensor) and t.shape == (n,) and t.dtype is dtype and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    _like(t, name, dtype, 1, index)  # says what is wrong
    raise ValueError(f"{name} must have {n} entries, got {t.shape[0]}")


def _output(out: torch.Tensor, name: str, shape, dtype: torch.dtype, index: int) -> torch.Tensor:
    _like(out, name, dtype, len(shape), index)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name} must be {dtype} {list(shape)}")
    return out


# ----------------------------------------------------------------------- norm
def awq_norm(h: torch.Tensor, weight: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
             bias: Optional[torch.Tensor] = None, post_weight: Optional[torch.Tensor] = None,
             post_bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
             gate_rows: Optional[torch.Tensor] = None, scale: float = 1.0, kind: str = "rms", eps: float = 1e-5,
             quantize: bool = False, h_out: Optional[torch.Tensor] = None) -> dict:
    """Ends a block and begins the next: with y (the block's output, fp16 [T][N]) the residual stream h
    (fp16 or fp32 [T][N]) becomes h + scale * gate * P(y), P the norm by post_weight and post_bias
    where given; with weight (fp16 [N]) x is the norm of that, or of h without y, by weight and bias.
    gate is fp16 [N], [T][N], or [rows][N] with gate_rows (int32 [T]: each token's row; one outside adds
    nothing).  kind "rms" or "layer".  Rows of h and y may be strided.

    Returns a dict: "h", the new residual stream (with y; in h_out where given, which may be h itself);
    "x" (with weight), fp16, or with quantize (rms, no bias) the rows in 8 bits that awq_gemm_i8
    takes as x and x_scales: int8 "x" and fp32 "scales"."""
    T, N, h_stride = _matrix(h, "h", _FLOATS, -1)
    index = h.get_device()
    y_stride = gates = 0
    h_ptr = y_ptr = x_ptr = scales_ptr = gate_ptr = rows_ptr = w_ptr = b_ptr = pw_ptr = pb_ptr = None
    out = {}
    if y is not None:
        Ty, Ny, y_stride = _matrix(y, "y", (_F16,), index)
        if Ty != T or Ny != N:
            raise ValueError(f"y must be [{T}][{N}], got {tuple(y.shape)}")
        y_ptr = y.data_ptr()
        if h_out is None:
            h_out = torch.empty_like(h) if h_stride == N else h.new_empty((T, N))
        else:
            _output(h_out, "h_out", (T, N), h.dtype, index)
        out["h"] = h_out
        h_ptr = h_out.data_ptr()
        if post_weight is not None:
            pw_ptr = _vector(post_weight, "post_weight", _F16, N, index)
    elif h_out is not None or post_weight is not None:
        raise ValueError("h_out and post_weight are only for a call with y")
    if post_bias is not None:
        pb_ptr = _vector(post_bias, "post_bias", _F16, N, index)
    if gate is not None:
        if isinstance(gate, torch.Tensor) and gate.dim() == 1:
            gate_ptr, gates = _vector(gate, "gate", _F16, N, index), 1
        else:
            _like(gate, "gate", _F16, 2, index)
            gates = gate.shape[0]
            if gate.shape[1] != N:
                raise ValueError(f"gate must have {N} columns, got {gate.shape[1]}")
            gate_ptr = gate.data_ptr()
    if gate_rows is not None:
        rows_ptr = _vector(gate_rows, "gate_rows", _I32, T, index)
    if weight is not None:
        w_ptr = _vector(weight, "weight", _F16, N, index)
        x = out["x"] = (torch.empty_like(y) if y_stride == N and not quantize else
                        h.new_empty((T, N), dtype=_I8 if quantize else _F16))
        x_ptr = x.data_ptr()
        if quantize:
            scales = out["scales"] = h.new_empty(T, dtype=_F32)
            scales_ptr = scales.data_ptr()
    elif quantize:
        raise ValueError("quantize needs weight")
    if bias is not None:
        b_ptr = _vector(bias, "bias", _F16, N, index)
    if kind == "rms":
        layer = 0
    elif kind in NORM_KINDS:
        layer = 1
    else:
        raise ValueError(f"kind must be one of {NORM_KINDS}, got {kind!r}")
    _run(index, load().awq_norm, h.data_ptr(), h.element_size(), h_stride, y_ptr, y_stride, pw_ptr, pb_ptr, gate_ptr, rows_ptr,
         gates, scale, w_ptr, b_ptr, layer, eps, h_ptr, x_ptr, scales_ptr, T, N)
    return out


# --------------------------------------------------------------- rows in 8 bits
def awq_quantize_rows(x: torch.Tensor, s: Optional[torch.Tensor] = None):
    """The rows of x (fp16 [M][K], strided rows allowed), or of x / s (fp32 [K]), in 8 bits: int8 codes
    [M][K] and fp32 scales [M], a row standing for code * scale."""
    M, K, stride = _matrix(x, "x", (_F16,), -1)
    index = x.get_device()
    codes, scales = x.new_empty((M, K), dtype=_I8), x.new_empty(M, dtype=_F32)
    _run(index, load().awq_quantize_rows, x.data_ptr(), stride, None if s is None else _vector(s, "s", _F32, K, index), M, K,
         codes.data_ptr(), scales.data_ptr())
    return codes, scales


def awq_pack_i8(W: torch.Tensor, s: Optional[torch.Tensor] = None):
    """The rows of W (fp16 [N][K]), or of W * s (fp32 [K]), in 8 bits, as awq_gemm_i8 takes them."""
    _need(W, "W", torch.float16, 2)
    index = W.get_device()
    N, K = W.shape
    codes, scales = W.new_empty((N, K), dtype=_I8), W.new_empty(N, dtype=_F32)
    _run(index, load().awq_pack_i8, W.data_ptr(), None if s is None else _vector(s, "s", _F32, K, index), N, K, codes.data_ptr(),
         scales.data_ptr())
    return codes, scales


def awq_gemm_i8_workspace_bytes(M: int, N: int, K: int, quantized: bool) -> int:
    return int(load().awq_gemm_i8_workspace_bytes(M, N, K, int(bool(quantized))))


def awq_gemm_i8(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, x_scales: Optional[torch.Tensor] = None,
                s: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                dtype: torch.dtype = torch.float16, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[m][n] = x_scales[m] * scales[n] * sum_k x[m][k] * codes[n][k] in exact whole-number sums, fp16
    or fp32 [M][N] (dtype, or out's).  codes int8 [N][K] and scales fp32 [N] as awq_pack_i8's; x int8
    [M][K] with x_scales fp32 [M] (awq_quantize_rows, awq_norm), or fp16 [M][K], which is quantised on
    the way, divided by s (fp32 [K]) first where given."""
    quantized = x_scales is not None
    _need(x, "x", _I8 if quantized else _F16, 2)
    index = x.get_device()
    _like(codes, "codes", _I8, 2, index)
    M, K = x.shape
    N, Kw = codes.shape
    if Kw != K:
        raise ValueError(f"codes are of rows of {Kw}, x of {K}")
    if out is None:
        if dtype not in _FLOATS:
            raise TypeError(f"y must be float16 or float32, got {dtype}")
        out = x.new_empty((M, N), dtype=dtype)
    else:
        dtype = out.dtype if isinstance(out, torch.Tensor) and out.dtype in _FLOATS else _F16
        _output(out, "out", (M, N), dtype, index)
    lib = load()
    ws, ws_bytes, _keep = _scratch(workspace, lib.awq_gemm_i8_workspace_bytes(M, N, K, quantized), x.device)
    _run(index, lib.awq_gemm_i8, x.data_ptr(), _vector(x_scales, "x_scales", _F32, M, index) if quantized else None,
         None if s is None else _vector(s, "s", _F32, K, index), codes.data_ptr(), _vector(scales, "scales", _F32, N, index),
         out.data_ptr(), out.element_size(), M, N, K, ws, ws_bytes)
    return out


def awq_gemm_i8_kernel(M: int, N: int, K: int, quantized: bool = True) -> str:
    """The kernel awq_gemm_i8 launches for these sizes (a host-only dry run of its dispatch)."""
    buf = ctypes.create_string_buffer(160)
    check(load().awq_gemm_i8_kernel(M, N, K, int(bool(quantized)), buf, len(buf)))
    return buf.value.decode()


# ------------------------------------------------------------------- next token
def _setting(v, name: str, dtype: torch.dtype, n: int, index: int):
    """(pointer, value) of a setting: a vector with an entry for each row, or a number for all."""
    if isinstance(v, torch.Tensor):
        return _vector(v, name, dtype, n, index), 0
    if dtype is _I32 and not -2 ** 31 <= v < 2 ** 31:  # would wrap round
        raise ValueError(f"{name}={v} does not fit 32 bits")
    return None, v


def awq_sample(logits: torch.Tensor, u: torch.Tensor, temperature: Union[float, torch.Tensor] = 1.0,
               top_k: Union[int, torch.Tensor] = 0, top_p: Union[float, torch.Tensor] = 1.0,
               min_p: Union[float, torch.Tensor] = 0.0) -> dict:
    """One token of each row of logits (fp16 or fp32 [B][V], strided rows allowed) from the random
    numbers u (fp32 [B], in [0, 1)): softmax at the temperature (0: the largest logit), cut to the top_k
    largest (0: all), of those to the fewest largest with top_p of the weight (1: all), of those to the ones
    with at least min_p times the largest weight; the token is where the remaining weights' running
    share, in index order, first exceeds u.  Each setting is one number, or a tensor with one for each
    row (fp32; top_k int32).  Returns a dict: int32 "tokens" [B] (-1 where every logit is -inf or NaN)
    and fp32 "probs" [B], the token's share of the remaining weights."""
    B, V, stride = _matrix(logits, "logits", _FLOATS, -1)
    index = logits.get_device()
    t_ptr, t = _setting(temperature, "temperature", _F32, B, index)
    k_ptr, k = _setting(top_k, "top_k", _I32, B, index)
    p_ptr, p = _setting(top_p, "top_p", _F32, B, index)
    m_ptr, m = _setting(min_p, "min_p", _F32, B, index)
    tokens, probs = logits.new_empty(B, dtype=_I32), logits.new_empty(B, dtype=_F32)
    _run(index, load().awq_sample, logits.data_ptr(), logits.element_size(), stride, B, V, t_ptr, t, k_ptr, k, p_ptr, p, m_ptr, m,
         _vector(u, "u", _F32, B, index), tokens.data_ptr(), probs.data_ptr())
    return dict(tokens=tokens, probs=probs)


__all__ = [n for n in dir() if n.startswith("awq_")] + ["NORM_KINDS"]
