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

import contextlib
import math
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from . import _abi

_PREC = {"bf16": _abi.DSA_PREC_BF16, "mxfp8": _abi.DSA_PREC_MXFP8, "fp8": _abi.DSA_PREC_FP8}
_NAME = {v: n for n, v in _PREC.items()}


@dataclass
class PagedCache:
    """Pages of keys and, unless `v` is None, values.

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
            self.prec = _NAME[self.prec]
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
        t = torch.zeros(shape, dtype=dt, device=device or "cuda")
        if prec == "bf16":
            return t, None
        n = head_dim // 32 if prec == "mxfp8" else 1
        return t, torch.zeros(shape[:3] + (n,), dtype=torch.uint8, device=t.device)

    k, ks = pages()
    v, vs = pages() if values else (None, None)
    return PagedCache(k, ks, v, vs, prec)


def _on(device: torch.device):
    """The tensors' device as the current one, for the launch and its stream."""
    if torch.cuda.current_device() == device.index:
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _arg(t: Optional[torch.Tensor], name: str, device: torch.device, dtype, shape=None) -> Optional[int]:
    """Address of a contiguous tensor of this type and shape on this device."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the CUDA device")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() or None


def _tokens(t: Optional[torch.Tensor], name: str, device: torch.device, dtypes, heads: int, head_dim: int):
    """Address and token stride of a [tokens, heads, head_dim] tensor whose tokens may be apart."""
    if t is None:
        return None, 0
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the CUDA device")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")
    if t.dim() != 3 or t.shape[1:] != (heads, head_dim):
        raise ValueError(f"{name} must be [tokens, {heads}, {head_dim}], not {tuple(t.shape)}")
    if (t.stride(2) != 1 and head_dim > 1) or (t.stride(1) != head_dim and heads > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return t.data_ptr() or None, (t.stride(0) if t.shape[0] > 1 else 0)


def _cache_args(c: PagedCache):
    return (c.k.data_ptr(), c.k_scale.data_ptr() if c.k_scale is not None else None,
            c.v.data_ptr() if c.v is not None else None, c.v_scale.data_ptr() if c.v_scale is not None else None)


def _batch(cache: PagedCache, page_table: torch.Tensor, cu_seqlens_k: torch.Tensor,
           cu_seqlens_q: Optional[torch.Tensor] = None):
    """Addresses of the page table and the prefixes, and the number of sequences."""
    dev = cache.k.device
    if not cache.k.is_cuda:
        raise ValueError("tensors must live on the CUDA device")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [num_seqs, max_pages]")
    B = page_table.shape[0]
    table = _arg(page_table, "page_table", dev, torch.int32)
    ck = _arg(cu_seqlens_k, "cu_seqlens_k", dev, torch.int32, (B + 1,))
    cq = _arg(cu_seqlens_q, "cu_seqlens_q", dev, torch.int32, (B + 1,))
    return table, ck, cq, B


def _workspace(ws: Optional[torch.Tensor], need: int, device: torch.device) -> torch.Tensor:
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    _arg(ws, "ws", device, torch.uint8)
    return ws


def cache_workspace(device=None) -> torch.Tensor:
    """Device workspace for cache_write and cache_read (read_status reads it)."""
    return torch.empty(_abi.load().dsa_idx_cache_workspace_size(), dtype=torch.uint8, device=device or "cuda")


def cache_write(cache: PagedCache, k: torch.Tensor, v: Optional[torch.Tensor], cu_seqlens_q: torch.Tensor,
                cu_seqlens_k: torch.Tensor, page_table: torch.Tensor, scale_rule="nosat",
                k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = None) -> None:
    """Store the new tokens' rows in the cache's format (dsa_idx_cache_write).

    k, v [tokens, n_kv_heads, head_dim], fp32 or bf16 (views with a token
    stride are taken as they are); v None for a cache of keys alone.  With an
    8-bit cache, uint8 k and v are E4M3 codes in operand form (as preprocess
    gives them) and k_scale, v_scale their UE8M0 bytes."""
    from . import _check, _rule, _stream
    dev = cache.k.device
    table, ck, cq, B = _batch(cache, page_table, cu_seqlens_k, cu_seqlens_q)
    Hk, D = cache.n_kv_heads, cache.head_dim
    kinds = (torch.float32, torch.bfloat16) + ((torch.uint8,) if cache.prec != "bf16" else ())
    kp, kst = _tokens(k, "k", dev, kinds, Hk, D)
    vp, vst = _tokens(v, "v", dev, (k.dtype,), Hk, D)
    if (v is None) != (cache.v is None):
        raise ValueError("v and the cache's values must both be given or both be None")
    if v is not None and v.shape[0] != k.shape[0]:
        raise ValueError("k and v must have the same tokens")
    T = k.shape[0]
    ksp = vsp = None
    if k.dtype == torch.uint8:
        if k_scale is None or (v is not None and v_scale is None):
            raise ValueError("codes come with their scales")
        n = cache.k_scale.shape[3]
        ksp = _arg(k_scale, "k_scale", dev, torch.uint8, (T, Hk, n))
        vsp = _arg(v_scale, "v_scale", dev, torch.uint8, (T, Hk, n))
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale belong to uint8 codes")
    dt = {torch.float32: _abi.DSA_DTYPE_F32, torch.bfloat16: _abi.DSA_DTYPE_BF16,
          torch.uint8: _abi.DSA_DTYPE_OPERAND}[k.dtype]
    with _on(dev):
        ws = _workspace(ws, _abi.DSA_CACHE_WS_BYTES, dev)
        a = _cache_args(cache)
        code = _abi.load().dsa_idx_cache_write(
            kp, kst, ksp, vp, vst, vsp, dt, _rule(scale_rule), cq, ck, B, T, table, page_table.shape[1], a[0], a[1],
            a[2], a[3], cache.num_pages, cache.page_size, Hk, D, _PREC[cache.prec], ws.data_ptr(), ws.numel(), _stream())
    _check(code, "dsa_idx_cache_write")


def cache_read(cache: PagedCache, cu_seqlens_k: torch.Tensor, page_table: torch.Tensor, total_k: int, out_prec=None,
               out=None, ws: Optional[torch.Tensor] = None
               ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Every sequence's rows, packed (dsa_idx_cache_read).

    Returns (k, k_scale, v, v_scale): rows as stored, k [total_k, n_kv_heads,
    head_dim] and scales [total_k, n_kv_heads, head_dim/32 or 1] (None for
    bf16; v and v_scale None for a cache of keys alone), or with
    out_prec="bf16" the values as bfloat16 and no scales.  `out` is such a
    tuple to write into; rows behind the last sequence stay as they were."""
    from . import _check, _stream
    dev = cache.k.device
    table, ck, _, B = _batch(cache, page_table, cu_seqlens_k)
    if out_prec not in (None, "bf16", cache.prec):
        raise ValueError(f"out_prec must be None or 'bf16' for a {cache.prec} cache, not {out_prec!r}")
    deq = out_prec == "bf16" and cache.prec != "bf16"
    Hk, D = cache.n_kv_heads, cache.head_dim
    dt = torch.bfloat16 if deq or cache.prec == "bf16" else torch.uint8
    n = 0 if dt == torch.bfloat16 else cache.k_scale.shape[3]
    with _on(dev):
        if out is None:
            def rows():
                t = torch.empty((total_k, Hk, D), dtype=dt, device=dev)
                return t, (torch.empty((total_k, Hk, n), dtype=torch.uint8, device=dev) if n else None)
            k, ks = rows()
            v, vs = rows() if cache.v is not None else (None, None)
        else:
            k, ks, v, vs = out
            if k is None or (n and (ks is None or (v is not None and vs is None))):
                raise ValueError("out lacks a tensor of this result")
            if v is not None and cache.v is None:
                raise ValueError("the cache has no values")
        ws = _workspace(ws, _abi.DSA_CACHE_WS_BYTES, dev)
        a = _cache_args(cache)
        code = _abi.load().dsa_idx_cache_read(
            a[0], a[1], a[2], a[3], cache.num_pages, cache.page_size, Hk, D, _PREC[cache.prec], table,
            page_table.shape[1], ck, B, total_k, int(deq), _arg(k, "out k", dev, dt, (total_k, Hk, D)),
            _arg(ks, "out k_scale", dev, torch.uint8, (total_k, Hk, n)) if n else None,
            _arg(v, "out v", dev, dt, (total_k, Hk, D)),
            _arg(vs, "out v_scale", dev, torch.uint8, (total_k, Hk, n)) if n else None, ws.data_ptr(), ws.numel(),
            _stream())
    _check(code, "dsa_idx_cache_read")
    return k, ks, v, vs


def attention_workspace(total_q: int, num_seqs: int, max_seqlen_q: int, n_heads: int, n_kv_heads: int, head_dim: int,
                        topk_width: int = 0, device=None) -> torch.Tensor:
    """Device workspace (uint8, 256-byte aligned) for paged_attention."""
    n = _abi.load().dsa_idx_attention_workspace_size(total_q, num_seqs, max_seqlen_q, n_heads, n_kv_heads, head_dim,
                                                     topk_width)
    if n == 0:
        raise ValueError("invalid workspace sizes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def paged_attention(q: torch.Tensor, cache: PagedCache, cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor,
                    page_table: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int, sm_scale: Optional[float] = None,
                    topk_idx: Optional[torch.Tensor] = None, topk_len: Optional[torch.Tensor] = None,
                    return_lse: bool = False, out=None, ws: Optional[torch.Tensor] = None):
    """Attention of the new tokens over the cache (dsa_idx_paged_attention).

    q [tokens, n_heads, head_dim] bf16 (a view with a token stride is taken as
    it is).  topk_idx int32 [tokens, W] restricts every query to the listed
    positions (score_topk's rows), topk_len int32 [tokens] to a row's first
    entries.  sm_scale defaults to head_dim ** -0.5.  Returns out [tokens,
    n_heads, head_dim] bf16, or (out, lse fp32 [tokens, n_heads]); `out` is
    such a tensor (or pair) to write into: rows behind the last sequence stay
    as they were."""
    from . import _check, _stream
    if cache.v is None:
        raise ValueError("the cache has no values")
    dev = cache.k.device
    table, ck, cq, B = _batch(cache, page_table, cu_seqlens_k, cu_seqlens_q)
    if q.dim() != 3:
        raise ValueError("q must be [tokens, n_heads, head_dim]")
    T, H, D = q.shape
    Hk = cache.n_kv_heads
    qp, qst = _tokens(q, "q", dev, (torch.bfloat16,), H, cache.head_dim)
    W = 0
    if topk_idx is not None:
        if topk_idx.dim() != 2:
            raise ValueError("topk_idx must be [tokens, width]")
        W = topk_idx.shape[1]
    elif topk_len is not None:
        raise ValueError("topk_len belongs to topk_idx")
    ip = _arg(topk_idx, "topk_idx", dev, torch.int32, (T, W))
    lp = _arg(topk_len, "topk_len", dev, torch.int32, (T,))
    lib = _abi.load()
    with _on(dev):
        lse = None
        if out is not None:
            out, lse = out if isinstance(out, (tuple, list)) else (out, None)
            if return_lse and lse is None:
                raise ValueError("out must be a pair (out, lse) with return_lse")
        else:
            out = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev)
            if return_lse:
                lse = torch.empty((T, H), dtype=torch.float32, device=dev)
        if ws is None:
            ws = attention_workspace(T, B, max_seqlen_q, H, Hk, D, W, dev)
        else:
            _arg(ws, "ws", dev, torch.uint8)
        a = _cache_args(cache)
        code = lib.dsa_idx_paged_attention(
            qp, qst, a[0], a[1], a[2], a[3], cache.num_pages, cache.page_size, H, Hk, D, _PREC[cache.prec], table,
            page_table.shape[1], cq, ck, B, T, max_seqlen_q, max_seqlen_k,
            1.0 / math.sqrt(D) if sm_scale is None else sm_scale, ip, lp, W,
            _arg(out, "out", dev, torch.bfloat16, (T, H, D)), _arg(lse, "lse", dev, torch.float32, (T, H)),
            ws.data_ptr(), ws.numel(), _stream())
    _check(code, "dsa_idx_paged_attention")
    return (out, lse) if return_lse else out
