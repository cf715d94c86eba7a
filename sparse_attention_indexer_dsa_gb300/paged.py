"""Paged cache: writing new tokens, reading them back, attention over the pages.

Binding of dsa_idx_cache_write, dsa_idx_cache_read and dsa_idx_paged_attention
(include/dsa_idx.h).  A serving step of a model with a sparse-attention
indexer is, per layer:

    dsa.cache_write(index_cache, k_op[:, None], None, cu_q, cu_k, table, k_scale=k_scale[:, None])
    dsa.cache_write(kv_cache, k, v, cu_q, cu_k, table)
    keys, key_scales, _, _ = dsa.cache_read(index_cache, cu_k, table, total_k)
    idx, _, lens = dsa.score_topk_kv(q_op, q_scale, keys[:, 0], key_scales[:, 0], w, cu_q, cu_k, ...)
    out = dsa.paged_attention(q, kv_cache, cu_q, cu_k, table, max_q, max_k, topk_idx=idx, topk_len=lens)
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from . import _abi

_PREC = {"bf16": _abi.DSA_PREC_BF16, "mxfp8": _abi.DSA_PREC_MXFP8, "fp8": _abi.DSA_PREC_FP8}
_NAME = {v: n for n, v in _PREC.items()}
_RULE = {"nosat": _abi.DSA_MX_SCALE_NOSAT, "floor": _abi.DSA_MX_SCALE_FLOOR}
_SOURCES = {torch.float32: _abi.DSA_DTYPE_F32, torch.bfloat16: _abi.DSA_DTYPE_BF16,
            torch.uint8: _abi.DSA_DTYPE_OPERAND}


def _rule(r) -> int:
    if isinstance(r, str):
        if r not in _RULE:
            raise ValueError(f"scale_rule must be 'nosat' or 'floor', not {r!r}")
        return _RULE[r]
    return r


def _error(code: int, where: str) -> Exception:
    from . import DsaError
    return DsaError(code, where)


@dataclass(frozen=True)
class PagedCache:
    """Pages of keys and, unless `v` is None, values: checked here, once, and so
    not to be replaced afterwards (a new handle costs next to nothing).

    k, v [num_pages, n_kv_heads, page_size, head_dim]: bfloat16 (prec "bf16")
    or uint8 E4M3 codes; k_scale, v_scale uint8 UE8M0 bytes
    [num_pages, n_kv_heads, page_size, head_dim/32] ("mxfp8") or
    [num_pages, n_kv_heads, page_size, 1] ("fp8"), None for "bf16"."""
    k: torch.Tensor
    k_scale: Optional[torch.Tensor]
    v: Optional[torch.Tensor]
    v_scale: Optional[torch.Tensor]
    prec: str = "bf16"

    def __post_init__(self):
        if self.prec not in _PREC:
            object.__setattr__(self, "prec", _NAME[self.prec])
        if self.k.dim() != 4:
            raise ValueError("pages are [num_pages, n_kv_heads, page_size, head_dim]")
        want = torch.bfloat16 if self.prec == "bf16" else torch.uint8
        if (self.v is None) != (self.v_scale is None) and self.prec != "bf16":
            raise ValueError("v and v_scale must both be given or both be None")
        for t, s in ((self.k, self.k_scale), (self.v, self.v_scale)):
            if t is None:
                continue
            if t.dtype != want or t.shape != self.k.shape or t.device != self.k.device or not t.is_contiguous():
                raise ValueError(f"{self.prec} pages are contiguous {want} tensors of one shape on one device")
            if self.prec == "bf16":
                if s is not None:
                    raise ValueError("bf16 pages have no scales")
                continue
            shape = t.shape[:3] + (t.shape[3] // 32 if self.prec == "mxfp8" else 1,)
            if s is None or s.dtype != torch.uint8 or s.shape != shape or s.device != t.device or not s.is_contiguous():
                raise ValueError(f"{self.prec} scales are a contiguous uint8 tensor {tuple(shape)} beside the pages")

    @property
    def num_pages(self) -> int:
        return self.k.shape[0]

    @property
    def n_kv_heads(self) -> int:
        return self.k.shape[1]

    @property
    def page_size(self) -> int:
        return self.k.shape[2]

    @property
    def head_dim(self) -> int:
        return self.k.shape[3]


def paged_cache(num_pages: int, page_size: int, n_kv_heads: int, head_dim: int, prec="bf16", values: bool = True,
                device=None) -> PagedCache:
    """A cache of zeros: keys and values, or keys alone (values=False, index keys)."""
    prec = _NAME.get(prec, prec)
    shape = (num_pages, n_kv_heads, page_size, head_dim)
    dt = torch.bfloat16 if prec == "bf16" else torch.uint8

    def pages():
        t = torch.zeros(shape, dtype=dt, device="cuda" if device is None else device)
        if prec == "bf16":
            return t, None
        n = head_dim // 32 if prec == "mxfp8" else 1
        return t, torch.zeros(shape[:3] + (n,), dtype=torch.uint8, device=t.device)

    k, ks = pages()
    v, vs = pages() if values else (None, None)
    return PagedCache(k, ks, v, vs, prec)


# The checks of one call run in a few microseconds of host time, a good part of
# a single-token call: one comparison per property, and the message only when one fails.
# (torch's own lookups behind its public functions; a torch without CUDA lacks them, and is imported all the same)
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_strided = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)


_modes = getattr(torch._C, "_len_torch_dispatch_stack", None)
_fills = torch.are_deterministic_algorithms_enabled


def _empty(shape: tuple, dtype, device: torch.device) -> torch.Tensor:
    """torch.empty; on the current device without the dispatch around the allocation (two of them before a launch:
    7.3 us of host time in place of 4.2), unless something wants to see or fill what is allocated.  The function that does
    it is not torch's public one: where it does not give what torch.empty gives, it is not called again."""
    global _strided
    if _strided is None or _modes is None or _modes() or _fills() or _current() != device.index:
        return torch.empty(shape, dtype=dtype, device=device)
    if len(shape) == 3:
        strides = (shape[1] * shape[2], shape[2], 1)
    elif len(shape) == 1:
        strides = (1,)
    else:
        strides, n = [1], 1
        for s in shape[:0:-1]:
            n *= s
            strides.append(n)
        strides = tuple(strides[::-1])
    try:
        t = _strided(shape, strides, dtype)
        if t.dtype is dtype and t.shape == shape:
            return t
    except (TypeError, AttributeError):   # another signature (what fails else, fails in torch.empty too)
        pass
    _strided = None
    return torch.empty(shape, dtype=dtype, device=device)


def _call(fn, device: torch.device, args) -> int:
    """The call with the tensors' device as the current one (changed only where it is not)."""
    if _current() == device.index:
        return fn(*args, _stream(device.index))
    with torch.cuda.device(device):
        return fn(*args, _stream(device.index))


def _refuse(t: torch.Tensor, name: str, device: torch.device, dtype, shape):
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the CUDA device")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _arg(t: Optional[torch.Tensor], name: str, device: torch.device, dtype, shape=None) -> Optional[int]:
    """Address of a contiguous tensor of this type and shape on this device."""
    if t is None:
        return None
    if t.dtype is not dtype or t.device != device or not t.is_contiguous() or (shape is not None and t.shape != shape):
        _refuse(t, name, device, dtype, shape)
    return t.data_ptr() or None


def _tokens(t: Optional[torch.Tensor], name: str, device: torch.device, dtypes, heads: int, head_dim: int):
    """Address and token stride of a [tokens, heads, head_dim] tensor whose tokens may be apart."""
    if t is None:
        return None, 0
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")
    if t.dim() != 3 or t.shape[1:] != (heads, head_dim):
        raise ValueError(f"{name} must be [tokens, {heads}, {head_dim}], not {tuple(t.shape)}")
    if t.device != device:
        _refuse(t, name, device, t.dtype, None)
    if t.is_contiguous():
        return t.data_ptr() or None, 0
    if t.stride(2) != 1 or (t.stride(1) != head_dim and heads > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    if t.shape[0] < 2:
        return t.data_ptr() or None, 0
    if t.stride(0) < heads * head_dim:   # (an expanded tensor's 0 would be taken for packed tokens)
        raise ValueError(f"{name}: tokens must not share memory (an expanded tensor is copied first)")
    return t.data_ptr() or None, t.stride(0)


def _pages(c: PagedCache):
    """Addresses of the pages and scales, device, and (num_pages, n_kv_heads, page_size, head_dim)."""
    k, ks, v, vs = c.k, c.k_scale, c.v, c.v_scale
    if not k.is_cuda:
        raise ValueError("tensors must live on the CUDA device")
    return ((k.data_ptr(), None if ks is None else ks.data_ptr(), None if v is None else v.data_ptr(),
             None if vs is None else vs.data_ptr()), k.device, k.shape)


def _table(page_table: torch.Tensor, device: torch.device):
    """Address of the page table, its width, the number of sequences."""
    if page_table.dim() != 2:
        raise ValueError("page_table must be [num_seqs, max_pages]")
    B, width = page_table.shape
    return _arg(page_table, "page_table", device, torch.int32), width, B


def cache_workspace(device=None) -> torch.Tensor:
    """Device workspace for cache_write and cache_read (read_status reads it)."""
    return torch.empty(_abi.load().dsa_idx_cache_workspace_size(), dtype=torch.uint8, device="cuda" if device is None else device)


def cache_write(cache: PagedCache, k: torch.Tensor, v: Optional[torch.Tensor], cu_seqlens_q: torch.Tensor,
                cu_seqlens_k: torch.Tensor, page_table: torch.Tensor, scale_rule="nosat",
                k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = None) -> None:
    """Store the new tokens' rows in the cache's format (dsa_idx_cache_write).

    k, v [tokens, n_kv_heads, head_dim], fp32 or bf16 (views with a token
    stride are taken as they are, tokens that share memory are refused); v None
    for a cache of keys alone.  With an 8-bit cache, uint8 k and v are E4M3 codes in operand form (as preprocess
    gives them) and k_scale, v_scale their UE8M0 bytes."""
    a, dev, (N, Hk, ps, D) = _pages(cache)
    table, width, B = _table(page_table, dev)
    T, dt = k.shape[0], k.dtype
    codes = dt is torch.uint8
    if codes and cache.prec == "bf16":
        raise ValueError("k: a bf16 cache stores fp32 or bf16 rows")
    kp, kst = _tokens(k, "k", dev, _SOURCES, Hk, D)
    vp, vst = _tokens(v, "v", dev, (dt,), Hk, D)
    if (v is None) != (cache.v is None):
        raise ValueError("v and the cache's values must both be given or both be None")
    if v is not None and v.shape[0] != T:
        raise ValueError("k and v must have the same tokens")
    ksp = vsp = None
    if codes:
        if k_scale is None or (v is not None and v_scale is None):
            raise ValueError("codes come with their scales")
        shape = (T, Hk, cache.k_scale.shape[3])
        ksp = _arg(k_scale, "k_scale", dev, torch.uint8, shape)
        vsp = _arg(v_scale, "v_scale", dev, torch.uint8, shape)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale belong to uint8 codes")
    cq = _arg(cu_seqlens_q, "cu_seqlens_q", dev, torch.int32, (B + 1,))
    ck = _arg(cu_seqlens_k, "cu_seqlens_k", dev, torch.int32, (B + 1,))
    if ws is None:
        ws = torch.empty(_abi.DSA_CACHE_WS_BYTES, dtype=torch.uint8, device=dev)
        wp = ws.data_ptr()
    else:
        wp = _arg(ws, "ws", dev, torch.uint8)
    code = _call(_abi.load().dsa_idx_cache_write, dev, (
        kp, kst, ksp, vp, vst, vsp, _SOURCES[dt], _rule(scale_rule), cq, ck, B, T, table, width, *a, N, ps, Hk, D,
        _PREC[cache.prec], wp, ws.numel()))
    if code:
        raise _error(code, "dsa_idx_cache_write")


def cache_read(cache: PagedCache, cu_seqlens_k: torch.Tensor, page_table: torch.Tensor, total_k: int, out_prec=None,
               out=None, ws: Optional[torch.Tensor] = None
               ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Every sequence's rows, packed (dsa_idx_cache_read).

    Returns (k, k_scale, v, v_scale): rows as stored, k [total_k, n_kv_heads,
    head_dim] and scales [total_k, n_kv_heads, head_dim/32 or 1] (None for
    bf16; v and v_scale None for a cache of keys alone), or with
    out_prec="bf16" the values as bfloat16 and no scales.  `out` is such a
    tuple to write into; rows behind the last sequence stay as they were."""
    a, dev, (N, Hk, ps, D) = _pages(cache)
    table, width, B = _table(page_table, dev)
    if out_prec not in (None, "bf16", cache.prec):
        raise ValueError(f"out_prec must be None or 'bf16' for a {cache.prec} cache, not {out_prec!r}")
    deq = out_prec == "bf16" and cache.prec != "bf16"
    values = deq or cache.prec == "bf16"
    dt = torch.bfloat16 if values else torch.uint8
    shape = (total_k, Hk, D)
    sshape = None if values else (total_k, Hk, cache.k_scale.shape[3])
    ck = _arg(cu_seqlens_k, "cu_seqlens_k", dev, torch.int32, (B + 1,))
    ks = v = vs = None
    if out is None:
        k = torch.empty(shape, dtype=dt, device=dev)
        if cache.v is not None:
            v = torch.empty(shape, dtype=dt, device=dev)
        if not values:
            ks = torch.empty(sshape, dtype=torch.uint8, device=dev)
            vs = None if v is None else torch.empty(sshape, dtype=torch.uint8, device=dev)
        kp, vp = k.data_ptr() or None, None if v is None else v.data_ptr()
    else:
        k, ks, v, vs = out
        if k is None or (not values and (ks is None or (v is not None and vs is None))):
            raise ValueError("out lacks a tensor of this result")
        if v is not None and cache.v is None:
            raise ValueError("the cache has no values")
        kp, vp = _arg(k, "out k", dev, dt, shape), _arg(v, "out v", dev, dt, shape)
    ksp = vsp = None
    if not values:
        ksp, vsp = _arg(ks, "out k_scale", dev, torch.uint8, sshape), _arg(vs, "out v_scale", dev, torch.uint8, sshape)
    if ws is None:
        ws = torch.empty(_abi.DSA_CACHE_WS_BYTES, dtype=torch.uint8, device=dev)
        wp = ws.data_ptr()
    else:
        wp = _arg(ws, "ws", dev, torch.uint8)
    code = _call(_abi.load().dsa_idx_cache_read, dev, (
        *a, N, ps, Hk, D, _PREC[cache.prec], table, width, ck, B, total_k, int(deq), kp, ksp, vp, vsp, wp, ws.numel()))
    if code:
        raise _error(code, "dsa_idx_cache_read")
    return k, ks, v, vs


def attention_workspace(total_q: int, num_seqs: int, max_seqlen_q: int, n_heads: int, n_kv_heads: int, head_dim: int,
                        topk_width: int = 0, device=None) -> torch.Tensor:
    """Device workspace (uint8, 256-byte aligned) for every paged_attention call of at most these sizes,
    with a list of any width if topk_width is not 0, without one if it is."""
    n = _abi.load().dsa_idx_attention_workspace_size(total_q, num_seqs, max_seqlen_q, n_heads, n_kv_heads, head_dim,
                                                     topk_width)
    if n == 0:
        raise ValueError("invalid workspace sizes")
    return torch.empty(n, dtype=torch.uint8, device="cuda" if device is None else device)


def paged_attention(q: torch.Tensor, cache: PagedCache, cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor,
                    page_table: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int, sm_scale: Optional[float] = None,
                    topk_idx: Optional[torch.Tensor] = None, topk_len: Optional[torch.Tensor] = None,
                    return_lse: bool = False, out=None, ws: Optional[torch.Tensor] = None):
    """Attention of the new tokens over the cache (dsa_idx_paged_attention).

    q [tokens, n_heads, head_dim] bf16 (a view with a token stride is taken as
    it is, tokens that share memory are refused).  topk_idx int32 [tokens, W]
    restricts every query to the listed positions (score_topk's rows), topk_len int32 [tokens] to a row's first
    entries.  sm_scale defaults to head_dim ** -0.5.  Returns out [tokens,
    n_heads, head_dim] bf16, or (out, lse fp32 [tokens, n_heads]); `out` is
    such a tensor (or pair) to write into: rows behind the last sequence stay
    as they were.  Forward only: no gradient is recorded.  `ws` from
    attention_workspace may be of a larger call; calls that may overlap need
    one each.  Without it the call allocates what it needs itself.  One plan
    serves a call: a long chunk and many single tokens are faster as two."""
    if cache.v is None:
        raise ValueError("the cache has no values")
    a, dev, (N, Hk, ps, D) = _pages(cache)
    table, width, B = _table(page_table, dev)
    if q.dim() != 3:
        raise ValueError("q must be [tokens, n_heads, head_dim]")
    T, H, _ = shape = q.shape
    qp, qst = _tokens(q, "q", dev, (torch.bfloat16,), H, D)
    cq = _arg(cu_seqlens_q, "cu_seqlens_q", dev, torch.int32, (B + 1,))
    ck = _arg(cu_seqlens_k, "cu_seqlens_k", dev, torch.int32, (B + 1,))
    W, ip, lp = 0, None, None
    if topk_idx is not None:
        if topk_idx.dim() != 2:
            raise ValueError("topk_idx must be [tokens, width]")
        W = topk_idx.shape[1]
        ip = _arg(topk_idx, "topk_idx", dev, torch.int32, (T, W))
        lp = _arg(topk_len, "topk_len", dev, torch.int32, (T,))
    elif topk_len is not None:
        raise ValueError("topk_len belongs to topk_idx")
    lse = lsep = None
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        op = out.data_ptr() or None
        if return_lse:
            lse = torch.empty((T, H), dtype=torch.float32, device=dev)
            lsep = lse.data_ptr() or None
    else:
        if isinstance(out, (tuple, list)):
            out, lse = out
        if return_lse and lse is None:
            raise ValueError("out must be a pair (out, lse) with return_lse")
        op = _arg(out, "out", dev, torch.bfloat16, shape)
        lsep = _arg(lse, "lse", dev, torch.float32, (T, H))
    if ws is None:
        n = _abi.load().dsa_idx_attention_call_workspace_size(T, B, max_seqlen_q, max_seqlen_k, H, Hk, D, ps,
                                                              _PREC[cache.prec], W)
        if n == 0:
            raise ValueError("invalid sizes")
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
    wp = _arg(ws, "ws", dev, torch.uint8)
    code = _call(_abi.load().dsa_idx_paged_attention, dev, (
        qp, qst, *a, N, ps, H, Hk, D, _PREC[cache.prec], table, width, cq, ck, B, T, max_seqlen_q, max_seqlen_k,
        D ** -0.5 if sm_scale is None else sm_scale, ip, lp, W, op, lsep, wp, ws.numel()))
    if code:
        raise _error(code, "dsa_idx_paged_attention")
    return (out, lse) if return_lse else out
