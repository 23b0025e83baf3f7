"""Torch-facing wrappers of the expert and key-value cache entry points.

As in api.py: each wrapper checks dtypes, devices and shapes, allocates outputs and
workspaces with torch on the inputs' device, and calls libawq on torch's current stream of
that device; all arithmetic happens in the library's HIP kernels.  Inputs on another device
than the first argument's are refused.

A decoding step makes many of these calls on little data, so the wrappers are kept short:
the device is switched only when it is not the current one, and a plan's arrays share one
allocation.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._lib import check, load
from .api import BITS, GROUP, _need, _ptr, packed_words

KV_BITS = (4, 8)               # code widths of a cache
KV_HEAD_DIMS = (64, 128, 256)  # channels of a head

_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle, without a Stream object


def _like(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int, index: int) -> None:
    """_need, on the given device."""
    if isinstance(t, torch.Tensor):
        if t.get_device() != index:
            raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
        if t.dtype is dtype and t.dim() == ndim and t.is_contiguous():
            return
    _need(t, name, dtype, ndim)  # says what is wrong


def _run(index: int, fn, *args) -> None:
    """fn(*args, stream) with the device current and its current stream; raises on a status."""
    if index == torch.cuda.current_device():
        check(fn(*args, _raw_stream(index)))
    else:
        with torch.cuda.device(index):
            check(fn(*args, _raw_stream(index)))


def _scratch(workspace: Optional[torch.Tensor], need: int, dev: torch.device):
    """(pointer, bytes) of the caller's workspace or a new one; the tensor too, to keep it."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not isinstance(workspace, torch.Tensor) or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


# --------------------------------------------------------------------- experts
def awq_moe_workspace_bytes(T: int, E: int, top_k: int) -> int:
    return int(load().awq_moe_workspace_bytes(T, E, top_k))


def _int_arrays(dev: torch.device, *sizes: int):
    """int32 arrays of these sizes in one allocation, each 16-byte aligned."""
    pieces = []
    for n in sizes:
        pieces.append(n)
        if n % 4:
            pieces.append(4 - n % 4)  # padding
    parts = torch.empty(sum(pieces), dtype=torch.int32, device=dev).split_with_sizes(pieces)
    if len(parts) == len(sizes):
        return parts
    out, i = [], 0
    for n in sizes:
        out.append(parts[i])
        i += 2 if n % 4 else 1
    return out


def _plan_workspace(T: int, E: int, top_k: int) -> int:
    need = load().awq_moe_workspace_bytes(T, E, top_k)
    if need == 0:
        raise ValueError(f"unsupported sizes for a plan: T={T}, E={E}, top_k={top_k}")
    return need


def awq_moe_plan(experts: torch.Tensor, num_experts: int) -> dict:
    """The plan of given choices (int32 [T][top_k]; an id outside [0, num_experts) drops the
    pair): offsets [E+1], rows and pos [T*top_k] as awq_gemm_grouped and awq_moe_combine take.  They
    share one allocation, which any of them keeps alive whole (as do awq_moe_route's results)."""
    _need(experts, "experts", torch.int32, 2)
    T, top_k = experts.shape
    need = _plan_workspace(T, num_experts, top_k)
    R = T * top_k
    rows, pos, offsets, ws = _int_arrays(experts.device, R, R, num_experts + 1, need // 4)
    _run(experts.get_device(), load().awq_moe_plan, experts.data_ptr(), T, num_experts, top_k, offsets.data_ptr(),
         rows.data_ptr(), pos.data_ptr(), ws.data_ptr(), need)
    return dict(offsets=offsets, rows=rows, pos=pos)


def awq_moe_route(logits: torch.Tensor, top_k: int, renormalize: bool = True) -> dict:
    """Each token's top_k experts (int32 [T][top_k], largest logit first, the lower index first
    where equal), their softmax weights (fp32 [T][top_k]; over all experts, or over the chosen
    ones with renormalize) and the plan (offsets, rows, pos).  logits: fp16 or fp32 [T][E]; one
    of -inf or NaN is never chosen (expert -1, weight 0 where too few are left)."""
    half = isinstance(logits, torch.Tensor) and logits.dtype == torch.float16
    _need(logits, "logits", torch.float16 if half else torch.float32, 2)
    T, E = logits.shape
    if not 1 <= top_k <= E:
        raise ValueError(f"top_k={top_k} outside [1, {E}]")
    need = _plan_workspace(T, E, top_k)
    R = T * top_k
    experts, weights, rows, pos, offsets, ws = _int_arrays(logits.device, R, R, R, R, E + 1, need // 4)
    _run(logits.get_device(), load().awq_moe_route, logits.data_ptr(), 2 if half else 4, T, E, top_k,
         int(bool(renormalize)), experts.data_ptr(), weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(),
         pos.data_ptr(), ws.data_ptr(), need)
    return dict(experts=experts.view(T, top_k), weights=weights.view(torch.float32).view(T, top_k), offsets=offsets,
                rows=rows, pos=pos)


def awq_gemm_grouped_workspace_bytes(R: int, K: int, scaled: bool) -> int:
    return int(load().awq_gemm_grouped_workspace_bytes(R, K, int(bool(scaled))))


def awq_gemm_grouped(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                     offsets: torch.Tensor, rows: Optional[torch.Tensor] = None, top_k: int = 1,
                     s: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, group: int = GROUP,
                     bits: Optional[int] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Row i of the ragged batch times the matrix of its expert e (offsets[e] <= i < offsets[e+1]):
    y fp16 [R][N].  packed int32 [E][N][words], scales fp16 [E][N][G], zeros uint8 [E][N][ceil(G/2)].
    Row i reads x[rows[i] / top_k] (rows int32 [R], as a plan's), or x[i] without rows; with s
    (fp32 [E][K]) it is divided by s[e] first: for few rows (R <= 5 E or 16, and at most 2048)
    kept to 22 bits, else rounded to fp16 as awq_scale_input does.  Rows from offsets[E] on
    are left as they were (in a new `out`: unset)."""
    _need(x, "x", torch.float16, 2)
    index = x.get_device()
    _like(packed, "packed", torch.int32, 3, index)
    _like(scales, "scales", torch.float16, 3, index)
    _like(zeros, "zeros", torch.uint8, 3, index)
    _like(offsets, "offsets", torch.int32, 1, index)
    x_rows, K = x.shape
    E, N, words = packed.shape
    G = K // group
    if bits is None:
        bits = next((b for b in BITS if words == packed_words(K, b)), None)
        if bits is None:
            raise ValueError(f"packed {tuple(packed.shape)} matches no format for K={K}")
    if words != packed_words(K, bits) or scales.shape != (E, N, G) or zeros.shape != (E, N, (G + 1) // 2):
        raise ValueError("packed/scales/zeros do not match x's K")
    if offsets.shape[0] != E + 1:
        raise ValueError(f"offsets must have E + 1 = {E + 1} entries")
    R, need = x_rows, 0
    if rows is not None:
        _like(rows, "rows", torch.int32, 1, index)
        R = rows.shape[0]
    lib = load()
    if s is not None:
        _like(s, "s", torch.float32, 2, index)
        if s.shape != (E, K):
            raise ValueError("s must be float32 [E][K]")
        need = lib.awq_gemm_grouped_workspace_bytes(R, K, 1)
    if out is None:
        out = x.new_empty((R, N))
    else:
        _like(out, "out", torch.float16, 2, index)
        if out.shape != (R, N):
            raise ValueError("out must be fp16 [R][N]")
    ws, ws_bytes, _keep = _scratch(workspace, need, x.device)
    _run(index, lib.awq_gemm_grouped, x.data_ptr(), x_rows, _ptr(rows), top_k, offsets.data_ptr(), _ptr(s),
         packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(), out.data_ptr(), R, E, N, K, group, bits, ws, ws_bytes)
    return out


def awq_gemm_grouped_kernel(R: int, E: int, N: int, K: int, bits: int = 4, group: int = GROUP) -> str:
    """The kernel awq_gemm_grouped launches for R rows over E experts of N x K (a host-only dry run
    of its dispatch: template arguments, block and grid)."""
    buf = ctypes.create_string_buffer(160)
    check(load().awq_gemm_grouped_kernel(R, E, N, K, group, bits, buf, len(buf)))
    return buf.value.decode()


def awq_moe_combine(y: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t] = sum_j weights[t][j] y[pos[t * top_k + j]] (fp32 sums, fp16 [T][N]); pairs with
    pos outside y add nothing.  weights fp32 [T][top_k], pos int32 [T*top_k]."""
    _need(y, "y", torch.float16, 2)
    index = y.get_device()
    _like(pos, "pos", torch.int32, 1, index)
    _like(weights, "weights", torch.float32, 2, index)
    R, N = y.shape
    T, top_k = weights.shape
    if pos.shape[0] != T * top_k:
        raise ValueError("pos must have T * top_k entries")
    if out is None:
        out = y.new_empty((T, N))
    else:
        _like(out, "out", torch.float16, 2, index)
        if out.shape != (T, N):
            raise ValueError("out must be fp16 [T][N]")
    _run(index, load().awq_moe_combine, y.data_ptr(), R, pos.data_ptr(), weights.data_ptr(), T, top_k, N,
         out.data_ptr())
    return out


# ----------------------------------------------------------- key-value cache
def empty_kv_cache(pages: int, heads: int, head_dim: int, page: int = 16, bits: int = 4, device="cuda") -> dict:
    """A paged cache: k_codes and v_codes int32 [pages][heads][page][head_dim*bits/32], k_params
    and v_params fp16 [pages][heads][page][2] (scale, zero point), and its code width `bits`."""
    if bits not in KV_BITS:
        raise ValueError(f"bits must be one of {KV_BITS}, got {bits}")
    if head_dim not in KV_HEAD_DIMS:
        raise ValueError(f"head_dim must be one of {KV_HEAD_DIMS}, got {head_dim}")
    if page < 16 or page > 1024 or page & (page - 1):
        raise ValueError(f"page must be a power of two in [16, 1024], got {page}")
    codes = lambda: torch.empty((pages, heads, page, head_dim * bits // 32), dtype=torch.int32, device=device)  # noqa: E731
    params = lambda: torch.empty((pages, heads, page, 2), dtype=torch.float16, device=device)  # noqa: E731
    return dict(k_codes=codes(), k_params=params(), v_codes=codes(), v_params=params(), bits=bits)


def _cache_args(cache: dict, head_dim: int, index: int):
    """The four arrays' pointers and (pages, heads, page, bits) of a cache of heads of head_dim channels."""
    kc, kp, vc, vp, bits = cache["k_codes"], cache["k_params"], cache["v_codes"], cache["v_params"], cache["bits"]
    if bits not in KV_BITS:
        raise ValueError(f"bits must be one of {KV_BITS}, got {bits}")
    _like(kc, "k_codes", torch.int32, 4, index)
    _like(kp, "k_params", torch.float16, 4, index)
    _like(vc, "v_codes", torch.int32, 4, index)
    _like(vp, "v_params", torch.float16, 4, index)
    shape, params = kc.shape, kp.shape
    pages, heads, page, words = shape
    if vc.shape != shape or vp.shape != params or params != (pages, heads, page, 2):
        raise ValueError("k_codes, k_params, v_codes and v_params are not of one cache")
    if words * 32 != head_dim * bits:
        raise ValueError(f"the cache's rows of {words} words do not hold {bits}-bit heads of {head_dim}")
    return (kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr()), pages, heads, page, bits


def _rows(t: torch.Tensor, name: str):
    """(T, H, D, elements from one token to the next) of fp16 [T][H][D] whose rows are contiguous
    within a token; any stride between tokens (a single token has no next)."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.float16 and t.dim() == 3):
        _need(t, name, torch.float16, 3)
    T, H, D = t.shape
    token, head, channel = t.stride()
    if channel != 1 or (H > 1 and head != D):
        raise ValueError(f"{name} must be contiguous within each token (heads, then channels)")
    return T, H, D, token if T > 1 else H * D


def awq_kv_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: dict) -> dict:
    """Quantises T tokens' keys and values (fp16 [T][heads][head_dim]; slices of a fused q/k/v
    product need no copy) into their slots (int32 [T], page number * page + place; one outside
    the cache, such as -1 for padding, is not written).  Returns the cache."""
    T, H, D, k_stride = _rows(k, "k")
    v_stride = _rows(v, "v")[3]
    index = k.get_device()
    _like(slots, "slots", torch.int32, 1, index)
    if v.shape != k.shape or v.get_device() != index or slots.shape[0] != T:
        raise ValueError("k and v must be fp16 [T][heads][head_dim] on one device, and slots int32 [T]")
    arrays, pages, heads, page, bits = _cache_args(cache, D, index)
    if heads != H:
        raise ValueError(f"k has {H} heads, the cache {heads}")
    _run(index, load().awq_kv_write, k.data_ptr(), v.data_ptr(), k_stride, v_stride, slots.data_ptr(),
         *arrays, T, H, D, pages, page, bits)
    return cache


def awq_kv_read(cache: dict, slots: torch.Tensor, head_dim: int):
    """The keys and values of T slots (int32 [T]), dequantised: two fp16 [T][heads][head_dim]; 0
    for a slot outside the cache."""
    _need(slots, "slots", torch.int32, 1)
    index = slots.get_device()
    arrays, pages, H, page, bits = _cache_args(cache, head_dim, index)
    T = slots.shape[0]
    k = cache["k_params"].new_empty((T, H, head_dim))
    v = k.new_empty((T, H, head_dim))
    _run(index, load().awq_kv_read, *arrays, slots.data_ptr(), k.data_ptr(), v.data_ptr(), T, H, head_dim, pages, page,
         bits)
    return k, v


def awq_kv_attention_workspace_bytes(B: int, Hq: int, Hkv: int, head_dim: int, bits: int, max_len: int) -> int:
    return int(load().awq_kv_attention_workspace_bytes(B, Hq, Hkv, head_dim, bits, max_len))


def awq_kv_attention(q: torch.Tensor, cache: dict, page_table: torch.Tensor, lengths: torch.Tensor,
                     scale: Optional[float] = None, max_len: int = 0, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of one new token of each sequence over the cache: fp16 [B][Hq][head_dim].
    q fp16 [B][Hq][head_dim] (a slice of a fused product needs no copy), page_table int32
    [B][width] (page of each run of `page` tokens; one outside the cache counts as absent),
    lengths int32 [B] (0: the output row is 0), scale 1/sqrt(head_dim) unless given, max_len a
    bound on the lengths (0: the table's width), workspace uint8 of
    awq_kv_attention_workspace_bytes bytes (allocated unless given)."""
    B, Hq, D, q_stride = _rows(q, "q")
    index = q.get_device()
    _like(page_table, "page_table", torch.int32, 2, index)
    _like(lengths, "lengths", torch.int32, 1, index)
    arrays, pages, Hkv, page, bits = _cache_args(cache, D, index)
    if page_table.shape[0] != B or lengths.shape[0] != B:
        raise ValueError("page_table must be int32 [B][width] and lengths int32 [B]")
    if Hkv < 1 or Hq % Hkv:
        raise ValueError(f"q's {Hq} heads are not a multiple of the cache's {Hkv}")
    if max_len < 0:
        raise ValueError(f"max_len must be >= 0, got {max_len}")
    if out is None:
        out = q.new_empty((B, Hq, D))
    else:
        _like(out, "out", torch.float16, 3, index)
        if out.shape != q.shape:
            raise ValueError("out must be fp16 [B][Hq][head_dim]")
    width = page_table.shape[1]
    bound = min(max_len, width * page) if max_len else width * page
    lib = load()
    ws, ws_bytes, _keep = _scratch(workspace, lib.awq_kv_attention_workspace_bytes(B, Hq, Hkv, D, bits, bound), q.device)
    _run(index, lib.awq_kv_attention, q.data_ptr(), q_stride, *arrays, page_table.data_ptr(), width,
         lengths.data_ptr(), out.data_ptr(), B, Hq, Hkv, D, pages, page, bits, D ** -0.5 if scale is None else scale,
         max_len, ws, ws_bytes)
    return out


__all__ = [n for n in dir() if n.startswith("awq_")] + ["empty_kv_cache", "KV_BITS", "KV_HEAD_DIMS"]
