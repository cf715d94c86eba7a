"""A paged cache of bounded length: the attention weight of its rows, the rows that stay, their moving together.

Binding of dsa_idx_cache_weigh, dsa_idx_evict_select and dsa_idx_cache_compact
(include/dsa_idx.h).  Per layer, with weights = dsa.paged_weights(cache) kept
beside the cache:

    out, lse = dsa.paged_attention(q, cache, cu_q, cu_k, table, max_q, max_k, return_lse=True)
    dsa.cache_weigh(cache, weights, q, lse, cu_q, cu_k, table, max_q, max_k)
    # where sequences have outgrown the budget
    kept, kept_len = dsa.evict_select(weights, cu_k, table, budget, max_k, sinks=4, recent=256)
    dsa.cache_compact(cache, kept, kept_len, table, weights=weights)

after which a sequence has kept_len cached rows.  A rotated row keeps the
position that it was written with, so nothing has to be turned again.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _abi
from .paged import _PREC, PagedCache, _arg, _call, _empty, _error, _pages, _table, _tokens


def paged_weights(cache: PagedCache) -> torch.Tensor:
    """Weights of a cache's rows, zeros: fp32 [num_pages, n_kv_heads, page_size]."""
    return torch.zeros(cache.k.shape[:3], dtype=torch.float32, device=cache.k.device)


def weigh_workspace(total_q: int, num_seqs: int, max_seqlen_q: int, n_heads: int, n_kv_heads: int, head_dim: int,
                    device=None) -> torch.Tensor:
    """Device workspace (uint8, 256-byte aligned) for every cache_weigh call of at most these sizes."""
    n = _abi.load().dsa_idx_weigh_workspace_size(total_q, num_seqs, max_seqlen_q, n_heads, n_kv_heads, head_dim)
    if n == 0:
        raise ValueError("invalid workspace sizes")
    return torch.empty(n, dtype=torch.uint8, device="cuda" if device is None else device)


def cache_weigh(cache: PagedCache, weights: torch.Tensor, q: torch.Tensor, lse: torch.Tensor, cu_seqlens_q: torch.Tensor,
                cu_seqlens_k: torch.Tensor, page_table: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int,
                sm_scale: Optional[float] = None, ws: Optional[torch.Tensor] = None) -> None:
    """Add the new tokens' attention weights to the rows that they see (dsa_idx_cache_weigh).

    weights fp32 [num_pages, n_kv_heads, page_size] (paged_weights) is updated
    in place: rows of earlier tokens gather, rows of the new tokens begin at 0.
    q [tokens, n_heads, head_dim] bf16 (a view with a token stride is taken as
    it is) and the other arguments as paged_attention took them, lse fp32
    [tokens, n_heads] as it returned it over every visible key.  A cache of
    keys alone will do.  Sequences of a call must not share pages."""
    a, dev, (N, Hk, ps, D) = _pages(cache)
    table, width, B = _table(page_table, dev)
    if q.dim() != 3:
        raise ValueError("q must be [tokens, n_heads, head_dim]")
    T, H, _ = q.shape
    qp, qst = _tokens(q, "q", dev, (torch.bfloat16,), H, D)
    lp = _arg(lse, "lse", dev, torch.float32, (T, H))
    wt = _arg(weights, "weights", dev, torch.float32, (N, Hk, ps))
    cq = _arg(cu_seqlens_q, "cu_seqlens_q", dev, torch.int32, (B + 1,))
    ck = _arg(cu_seqlens_k, "cu_seqlens_k", dev, torch.int32, (B + 1,))
    if ws is None:
        ws = weigh_workspace(T, B, max_seqlen_q, H, Hk, D, dev)
    code = _call(_abi.load().dsa_idx_cache_weigh, dev, (
        qp, qst, lp, a[0], a[1], wt, N, ps, H, Hk, D, _PREC[cache.prec], table, width, cq, ck, B, T, max_seqlen_q,
        max_seqlen_k, D ** -0.5 if sm_scale is None else sm_scale, _arg(ws, "ws", dev, torch.uint8), ws.numel()))
    if code:
        raise _error(code, "dsa_idx_cache_weigh")


def _status_ws(ws: Optional[torch.Tensor], dev: torch.device):
    """Address and size of a workspace that holds the status alone, and the tensor."""
    if ws is None:
        ws = _empty((_abi.DSA_CACHE_WS_BYTES,), torch.uint8, dev)
    return _arg(ws, "ws", dev, torch.uint8), ws.numel(), ws


def evict_select(weights: torch.Tensor, cu_seqlens_k: torch.Tensor, page_table: torch.Tensor, budget: int,
                 max_seqlen_k: int, sinks: int = 0, recent: int = 0, shared: bool = False, out=None,
                 ws: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The rows of each sequence that stay (dsa_idx_evict_select).

    All rows where there are at most `budget`, else the first `sinks`, the last
    `recent` and the heaviest of the others, ties to the lower position; each
    head on its own, or with shared=True one choice by the heads' summed
    weights.  Returns (kept int32 [num_seqs, n_kv_heads or 1, budget],
    ascending, then -1, kept_len int32 [num_seqs]); `out` is such a pair to
    write into.  `ws` from cache_workspace."""
    if budget >> 31 or max_seqlen_k >> 31 or sinks >> 31 or recent >> 31:   # (ctypes would drop the upper bits)
        raise ValueError("budget, max_seqlen_k, sinks and recent must be in [0, 2^31)")
    if weights.dim() != 3:
        raise ValueError("weights must be [num_pages, n_kv_heads, page_size]")
    if not weights.is_cuda:
        raise ValueError("weights must live on the CUDA device")
    dev = weights.device
    N, Hk, ps = weights.shape
    wt = _arg(weights, "weights", dev, torch.float32)
    table, width, B = _table(page_table, dev)
    ck = _arg(cu_seqlens_k, "cu_seqlens_k", dev, torch.int32, (B + 1,))
    if budget < 1:
        raise ValueError("budget must be at least 1")
    shape = (B, 1 if shared else Hk, budget)
    if out is None:
        kept, kept_len = _empty(shape, torch.int32, dev), _empty((B,), torch.int32, dev)
    else:
        kept, kept_len = out
    kp, lp = _arg(kept, "kept", dev, torch.int32, shape), _arg(kept_len, "kept_len", dev, torch.int32, (B,))
    wp, n, ws = _status_ws(ws, dev)
    code = _call(_abi.load().dsa_idx_evict_select, dev, (
        wt, N, ps, Hk, table, width, ck, B, max_seqlen_k, budget, sinks, recent, int(shared), kp, lp, wp, n))
    if code:
        raise _error(code, "dsa_idx_evict_select")
    return kept, kept_len


def cache_compact(cache: PagedCache, kept: torch.Tensor, kept_len: torch.Tensor, page_table: torch.Tensor,
                  weights: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> None:
    """Move the kept rows of every sequence to its first positions, in place (dsa_idx_cache_compact).

    kept int32 [num_seqs, n_kv_heads or 1, width] and kept_len int32 [num_seqs]
    as evict_select gives them; keys, values, scales and, unless None, weights
    (fp32 [num_pages, n_kv_heads, page_size]) move together.  Sequences must
    not share pages.  `ws` from cache_workspace."""
    a, dev, (N, Hk, ps, D) = _pages(cache)
    table, width, B = _table(page_table, dev)
    if kept.dim() != 3 or kept.shape[0] != B or kept.shape[1] not in (1, Hk):
        raise ValueError(f"kept must be [{B}, {Hk} or 1, width], not {tuple(kept.shape)}")
    kp, lp = _arg(kept, "kept", dev, torch.int32), _arg(kept_len, "kept_len", dev, torch.int32, (B,))
    wt = _arg(weights, "weights", dev, torch.float32, (N, Hk, ps))
    wp, n, ws = _status_ws(ws, dev)
    code = _call(_abi.load().dsa_idx_cache_compact, dev, (
        *a, wt, N, ps, Hk, D, _PREC[cache.prec], table, width, kp, lp, B, kept.shape[1], kept.shape[2], wp, n))
    if code:
        raise _error(code, "dsa_idx_cache_compact")
