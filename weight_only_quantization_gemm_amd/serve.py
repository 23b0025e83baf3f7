"""Torch-facing wrappers of the expert and key-value cache entry points.

As in api.py: each wrapper checks dtypes, devices and shapes, allocates outputs and
workspaces with torch on the inputs' device, and calls libawq on torch's current stream of
that device; all arithmetic happens in the library's HIP kernels.  Inputs on another device
than the first argument's are refused.
"""
from __future__ import annotations

from typing import Optional

import torch

from ._lib import check, load
from .api import BITS, GROUP, _need, _ptr, _stream, packed_words

KV_BITS = (4, 8)               # code widths of a cache
KV_HEAD_DIMS = (64, 128, 256)  # channels of a head
CACHE_KEYS = ("k_codes", "k_params", "v_codes", "v_params")


def _on(dev: torch.device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")


# --------------------------------------------------------------------- experts
def awq_moe_workspace_bytes(T: int, E: int, top_k: int) -> int:
    return int(load().awq_moe_workspace_bytes(T, E, top_k))


def _plan_buffers(T: int, E: int, top_k: int, dev: torch.device):
    need = awq_moe_workspace_bytes(T, E, top_k)
    if need == 0:
        raise ValueError(f"unsupported sizes for a plan: T={T}, E={E}, top_k={top_k}")
    ints = dict(dtype=torch.int32, device=dev)
    return (dict(offsets=torch.empty(E + 1, **ints), rows=torch.empty(T * top_k, **ints),
                 pos=torch.empty(T * top_k, **ints)), torch.empty(need, dtype=torch.uint8, device=dev), need)


def awq_moe_plan(experts: torch.Tensor, num_experts: int) -> dict:
    """The plan of given choices (int32 [T][top_k]; an id outside [0, num_experts) drops the
    pair): offsets [E+1], rows and pos [T*top_k] as awq_gemm_grouped and awq_moe_combine take."""
    _need(experts, "experts", torch.int32, 2)
    T, top_k = experts.shape
    plan, ws, need = _plan_buffers(T, num_experts, top_k, experts.device)
    with torch.cuda.device(experts.device):
        check(load().awq_moe_plan(experts.data_ptr(), T, num_experts, top_k, plan["offsets"].data_ptr(),
                                  plan["rows"].data_ptr(), plan["pos"].data_ptr(), ws.data_ptr(), need,
                                  _stream(experts.device)))
    return plan


def awq_moe_route(logits: torch.Tensor, top_k: int, renormalize: bool = True) -> dict:
    """Each token's top_k experts (int32 [T][top_k], largest logit first, the lower index first
    where equal), their softmax weights (fp32 [T][top_k]; over all experts, or over the chosen
    ones with renormalize) and the plan (offsets, rows, pos).  logits: fp16 or fp32 [T][E]; one
    of -inf or NaN is never chosen (expert -1, weight 0 where too few are left)."""
    half = isinstance(logits, torch.Tensor) and logits.dtype == torch.float16
    _need(logits, "logits", torch.float16 if half else torch.float32, 2)
    T, E = logits.shape
    dev = logits.device
    if not 1 <= top_k <= E:
        raise ValueError(f"top_k={top_k} outside [1, {E}]")
    plan, ws, need = _plan_buffers(T, E, top_k, dev)
    experts = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        check(load().awq_moe_route(logits.data_ptr(), 2 if half else 4, T, E, top_k, int(bool(renormalize)),
                                   experts.data_ptr(), weights.data_ptr(), plan["offsets"].data_ptr(),
                                   plan["rows"].data_ptr(), plan["pos"].data_ptr(), ws.data_ptr(), need, _stream(dev)))
    return dict(experts=experts, weights=weights, **plan)


def awq_gemm_grouped_workspace_bytes(R: int, K: int, scaled: bool) -> int:
    return int(load().awq_gemm_grouped_workspace_bytes(R, K, int(bool(scaled))))


def awq_gemm_grouped(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                     offsets: torch.Tensor, rows: Optional[torch.Tensor] = None, top_k: int = 1,
                     s: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, group: int = GROUP,
                     bits: Optional[int] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Row i of the ragged batch times the matrix of its expert e (offsets[e] <= i < offsets[e+1]):
    y fp16 [R][N].  packed int32 [E][N][words], scales fp16 [E][N][G], zeros uint8 [E][N][ceil(G/2)].
    Row i reads x[rows[i] / top_k] (rows int32 [R], as a plan's), or x[i] without rows; with s
    (fp32 [E][K]) it is divided by s[e] first, as awq_scale_input does.  Rows from offsets[E] on
    are left as they were (in a new `out`: unset)."""
    _need(x, "x", torch.float16, 2)
    _need(packed, "packed", torch.int32, 3)
    _need(scales, "scales", torch.float16, 3)
    _need(zeros, "zeros", torch.uint8, 3)
    _need(offsets, "offsets", torch.int32, 1)
    dev = x.device
    x_rows, K = x.shape
    E, N, words = packed.shape
    G = K // group
    if bits is None:
        bits = next((b for b in BITS if words == packed_words(K, b)), None)
        if bits is None:
            raise ValueError(f"packed {tuple(packed.shape)} matches no format for K={K}")
    if words != packed_words(K, bits) or tuple(scales.shape) != (E, N, G) or tuple(zeros.shape) != (E, N, (G + 1) // 2):
        raise ValueError("packed/scales/zeros do not match x's K")
    if offsets.shape[0] != E + 1:
        raise ValueError(f"offsets must have E + 1 = {E + 1} entries")
    if rows is not None:
        _need(rows, "rows", torch.int32, 1)
    R = x_rows if rows is None else rows.shape[0]
    if s is not None:
        _need(s, "s", torch.float32, 2)
        if tuple(s.shape) != (E, K):
            raise ValueError("s must be float32 [E][K]")
    if out is None:
        out = torch.empty((R, N), dtype=torch.float16, device=dev)
    else:
        _need(out, "out", torch.float16, 2)
        if tuple(out.shape) != (R, N):
            raise ValueError("out must be fp16 [R][N]")
    lib = load()
    need = lib.awq_gemm_grouped_workspace_bytes(R, K, 1) if s is not None else 0
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _on(dev, packed=packed, scales=scales, zeros=zeros, offsets=offsets, rows=rows, s=s, out=out, workspace=workspace)
    with torch.cuda.device(dev):
        check(lib.awq_gemm_grouped(x.data_ptr(), x_rows, _ptr(rows), top_k, offsets.data_ptr(), _ptr(s),
                                   packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(), out.data_ptr(), R, E, N, K,
                                   group, bits, _ptr(workspace),
                                   0 if workspace is None else workspace.numel() * workspace.element_size(),
                                   _stream(dev)))
    return out


def awq_moe_combine(y: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t] = sum_j weights[t][j] y[pos[t * top_k + j]] (fp32 sums, fp16 [T][N]); pairs with
    pos outside y add nothing.  weights fp32 [T][top_k], pos int32 [T*top_k]."""
    _need(y, "y", torch.float16, 2)
    _need(pos, "pos", torch.int32, 1)
    _need(weights, "weights", torch.float32, 2)
    R, N = y.shape
    T, top_k = weights.shape
    if pos.shape[0] != T * top_k:
        raise ValueError("pos must have T * top_k entries")
    if out is None:
        out = torch.empty((T, N), dtype=torch.float16, device=y.device)
    else:
        _need(out, "out", torch.float16, 2)
        if tuple(out.shape) != (T, N):
            raise ValueError("out must be fp16 [T][N]")
    _on(y.device, pos=pos, weights=weights, out=out)
    with torch.cuda.device(y.device):
        check(load().awq_moe_combine(y.data_ptr(), R, pos.data_ptr(), weights.data_ptr(), T, top_k, N, out.data_ptr(),
                                     _stream(y.device)))
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


def _cache_shape(cache: dict, head_dim: int, dev: torch.device):
    """(pages, heads, page, bits) of a cache whose heads have head_dim channels."""
    bits = cache["bits"]
    if bits not in KV_BITS:
        raise ValueError(f"bits must be one of {KV_BITS}, got {bits}")
    shape = cache["k_codes"].shape
    for name in CACHE_KEYS:
        t = cache[name]
        _need(t, name, torch.int32 if name.endswith("codes") else torch.float16, 4)
        if t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")
        if t.shape[:3] != shape[:3] or t.shape[3] != (head_dim * bits // 32 if name.endswith("codes") else 2):
            raise ValueError(f"{name} {tuple(t.shape)} does not match the cache's other arrays, or {bits}-bit heads "
                             f"of {head_dim}")
    return shape[0], shape[1], shape[2], bits


def _need_rows(t: torch.Tensor, name: str) -> None:
    """fp16 [T][H][D] whose rows are contiguous within a token; any stride between tokens."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (libawq has no CPU path)")
    if t.dtype != torch.float16:
        raise TypeError(f"{name} must be {torch.float16}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dims, got {tuple(t.shape)}")
    if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise ValueError(f"{name} must be contiguous within each token (heads, then channels)")


def _token_stride(t: torch.Tensor) -> int:
    """Elements from one token's rows to the next (a single token has no next)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def awq_kv_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: dict) -> dict:
    """Quantises T tokens' keys and values (fp16 [T][heads][head_dim]; slices of a fused q/k/v
    product need no copy) into their slots (int32 [T], page number * page + place; one outside
    the cache, such as -1 for padding, is not written).  Returns the cache."""
    _need_rows(k, "k")
    _need_rows(v, "v")
    _need(slots, "slots", torch.int32, 1)
    T, H, D = k.shape
    if v.shape != k.shape or slots.shape[0] != T:
        raise ValueError("k and v must be fp16 [T][heads][head_dim] and slots int32 [T]")
    dev = k.device
    pages, heads, page, bits = _cache_shape(cache, D, dev)
    if heads != H:
        raise ValueError(f"k has {H} heads, the cache {heads}")
    _on(dev, v=v, slots=slots)
    with torch.cuda.device(dev):
        check(load().awq_kv_write(k.data_ptr(), v.data_ptr(), _token_stride(k), _token_stride(v), slots.data_ptr(),
                                  cache["k_codes"].data_ptr(), cache["k_params"].data_ptr(),
                                  cache["v_codes"].data_ptr(), cache["v_params"].data_ptr(), T, H, D, pages, page,
                                  bits, _stream(dev)))
    return cache


def awq_kv_read(cache: dict, slots: torch.Tensor, head_dim: int):
    """The keys and values of T slots (int32 [T]), dequantised: two fp16 [T][heads][head_dim]; 0
    for a slot outside the cache."""
    _need(slots, "slots", torch.int32, 1)
    dev = slots.device
    pages, H, page, bits = _cache_shape(cache, head_dim, dev)
    T = slots.shape[0]
    k = torch.empty((T, H, head_dim), dtype=torch.float16, device=dev)
    v = torch.empty_like(k)
    with torch.cuda.device(dev):
        check(load().awq_kv_read(cache["k_codes"].data_ptr(), cache["k_params"].data_ptr(),
                                 cache["v_codes"].data_ptr(), cache["v_params"].data_ptr(), slots.data_ptr(),
                                 k.data_ptr(), v.data_ptr(), T, H, head_dim, pages, page, bits, _stream(dev)))
    return k, v


def awq_kv_attention_workspace_bytes(B: int, Hq: int, Hkv: int, head_dim: int, max_len: int) -> int:
    return int(load().awq_kv_attention_workspace_bytes(B, Hq, Hkv, head_dim, max_len))


def awq_kv_attention(q: torch.Tensor, cache: dict, page_table: torch.Tensor, lengths: torch.Tensor,
                     scale: Optional[float] = None, max_len: int = 0, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of one new token of each sequence over the cache: fp16 [B][Hq][head_dim].
    q fp16 [B][Hq][head_dim] (a slice of a fused product needs no copy), page_table int32
    [B][width] (page of each run of `page` tokens; one outside the cache counts as absent),
    lengths int32 [B] (0: the output row is 0), scale 1/sqrt(head_dim) unless given, max_len a
    bound on the lengths (0: the table's width), workspace uint8 of
    awq_kv_attention_workspace_bytes bytes (allocated unless given)."""
    _need_rows(q, "q")
    _need(page_table, "page_table", torch.int32, 2)
    _need(lengths, "lengths", torch.int32, 1)
    B, Hq, D = q.shape
    dev = q.device
    pages, Hkv, page, bits = _cache_shape(cache, D, dev)
    if page_table.shape[0] != B or lengths.shape[0] != B:
        raise ValueError("page_table must be int32 [B][width] and lengths int32 [B]")
    if Hq % Hkv:
        raise ValueError(f"q's {Hq} heads are not a multiple of the cache's {Hkv}")
    if max_len < 0:
        raise ValueError(f"max_len must be >= 0, got {max_len}")
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float16, device=dev)
    else:
        _need(out, "out", torch.float16, 3)
        if out.shape != q.shape:
            raise ValueError("out must be fp16 [B][Hq][head_dim]")
    width = page_table.shape[1]
    bound = min(max_len, width * page) if max_len else width * page
    lib = load()
    need = lib.awq_kv_attention_workspace_bytes(B, Hq, Hkv, D, bound)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _on(dev, page_table=page_table, lengths=lengths, out=out, workspace=workspace)
    with torch.cuda.device(dev):
        check(lib.awq_kv_attention(q.data_ptr(), _token_stride(q), cache["k_codes"].data_ptr(),
                                   cache["k_params"].data_ptr(), cache["v_codes"].data_ptr(),
                                   cache["v_params"].data_ptr(), page_table.data_ptr(), width, lengths.data_ptr(),
                                   out.data_ptr(), B, Hq, Hkv, D, pages, page, bits,
                                   D ** -0.5 if scale is None else scale, max_len, _ptr(workspace),
                                   0 if workspace is None else workspace.numel() * workspace.element_size(),
                                   _stream(dev)))
    return out


__all__ = [n for n in dir() if n.startswith("awq_")] + ["empty_kv_cache", "KV_BITS", "KV_HEAD_DIMS"]
