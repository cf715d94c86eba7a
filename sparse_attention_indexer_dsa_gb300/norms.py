"""Norms of queries and keys for each head with the position rotation, and their gradients.

Binding of dsa_idx_norm_rope and dsa_idx_norm_rope_backward (include/dsa_idx.h).
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import _abi
from .paged import _arg, _call, _empty, _error

_NORM = {"rms": _abi.DSA_NORM_RMS, "layer": _abi.DSA_NORM_LAYER}
_WEIGHTS = ("q_weight", "k_weight", "q_bias", "k_bias")
_DTYPE = {torch.float32: _abi.DSA_DTYPE_F32, torch.bfloat16: _abi.DSA_DTYPE_BF16}


class NormRopeGrads(NamedTuple):
    """Gradients of norm_rope's inputs; None for what the call does not have."""
    q: torch.Tensor
    k: Optional[torch.Tensor]
    q_weight: Optional[torch.Tensor]
    k_weight: Optional[torch.Tensor]
    q_bias: Optional[torch.Tensor]
    k_bias: Optional[torch.Tensor]


def _rows(t: torch.Tensor, name: str):
    """Address and token stride of a [tokens, heads, head_dim] tensor whose tokens may be apart."""
    if t.is_contiguous():
        return t.data_ptr() or None, 0
    T, H, D = t.shape
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != D and H > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    if T < 2:
        return t.data_ptr() or None, 0
    if s0 < H * D:   # (an expanded tensor's 0 would be taken for packed tokens)
        raise ValueError(f"{name}: tokens must not share memory (an expanded tensor is copied first)")
    return t.data_ptr() or None, s0


def _like(t: torch.Tensor, name: str, shape, dtype, device):
    """The same of a tensor that must be of this shape, type and device."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype} on {device}, not {tuple(t.shape)} {t.dtype} on {t.device}")
    return _rows(t, name)


def _inputs(q, k, positions, weights, norm, rope_dim, inv_freq):
    """Checks that forward and backward share; what they hand on."""
    if q.dim() != 3:
        raise ValueError("q must be [tokens, n_heads, head_dim]")
    shape, dev, dt = q.shape, q.device, q.dtype
    T, H, D = shape
    if not q.is_cuda:
        raise ValueError("q must live on the CUDA device")
    if dt not in _DTYPE:
        raise ValueError(f"q: unsupported dtype {dt}")
    if norm not in _NORM:
        raise ValueError(f"norm must be 'rms' or 'layer', not {norm!r}")
    qp, qst = _rows(q, "q")
    kp, kst, Hk = None, 0, 0
    if k is not None:
        if k.dim() != 3:
            raise ValueError(f"k must be [{T}, n_kv_heads, {D}], not {tuple(k.shape)}")
        Hk = k.shape[1]
        kp, kst = _like(k, "k", (T, Hk, D), dt, dev)
    R = D if rope_dim is None else rope_dim
    if R >> 31:   # (ctypes would drop the upper bits)
        raise ValueError("rope_dim must be a multiple of 8 in [0, head_dim]")
    pos = None
    if R:
        if positions is None:
            raise ValueError("positions are needed unless rope_dim is 0")
        pos = _arg(positions, "positions", dev, torch.int32, (T,))
    wt, wp = None, [None, None, None, None]
    for i, w in enumerate(weights):
        if w is not None:
            if wt is None:
                wt = w.dtype
                if wt not in _DTYPE:
                    raise ValueError(f"weights: unsupported dtype {wt}")
            if i & 1 and k is None:
                raise ValueError("k_weight and k_bias belong to k")
            wp[i] = _arg(w, _WEIGHTS[i], dev, wt, (D,))
    freq = None
    if inv_freq is not None:
        if len(inv_freq) != R // 2:
            raise ValueError(f"inv_freq must have rope_dim / 2 = {R // 2} values")
        freq = (ctypes.c_double * max(1, R // 2))(*[float(f) for f in inv_freq])
    return shape, dev, dt, Hk, (qp, qst, kp, kst), R, pos, wp, 0 if wt is None else _DTYPE[wt], freq


def norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: Optional[torch.Tensor],
              q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
              q_bias: Optional[torch.Tensor] = None, k_bias: Optional[torch.Tensor] = None, norm: str = "rms",
              eps: float = 1e-6, rope_dim: Optional[int] = None, rope_base: float = 10000.0,
              inv_freq: Optional[Sequence[float]] = None, rope_interleaved: bool = False,
              out_dtype: Optional[torch.dtype] = None, out=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Norm of each head's row, weights (and biases), then the rotation by its token's position (dsa_idx_norm_rope).

    q [tokens, n_heads, head_dim], k [tokens, n_kv_heads, head_dim] or None,
    fp32 or bf16 (views with a token stride, as slices of one projection, are
    taken as they are); positions int32 [tokens]; weights and biases [head_dim],
    fp32 or bf16, None: ones and zeros.  norm "rms", which takes no biases (none
    of its gradients would be theirs), or "layer".  rope_dim: the first
    dimensions of a head are rotated (default: all; 0: none), by rope_base or by
    the rope_dim / 2 host values inv_freq.  Returns (q_out, k_out or None)
    in out_dtype (default: q's); `out` is such a pair to write into, and may be
    (q, k) itself.  No gradient is recorded: norm_rope_backward gives it."""
    shape, dev, dt, Hk, rows, R, pos, wp, wt, freq = _inputs(q, k, positions, (q_weight, k_weight, q_bias, k_bias), norm,
                                                            rope_dim, inv_freq)
    T, H, D = shape
    if out is None:
        ot = dt if out_dtype is None else out_dtype
        if ot not in _DTYPE:
            raise ValueError(f"out_dtype: unsupported dtype {ot}")
        q_out, k_out = _empty((T, H, D), ot, dev), None
        qo, qost, ko, kost = q_out.data_ptr() or None, 0, None, 0
        if k is not None:
            k_out = _empty((T, Hk, D), ot, dev)
            ko = k_out.data_ptr() or None
    else:
        q_out, k_out = out
        ot = q_out.dtype
        if out_dtype not in (None, ot):
            raise ValueError("out has another dtype than out_dtype")
        if (k is None) != (k_out is None):
            raise ValueError("out must be a pair (q_out, k_out), k_out None where k is")
        if ot not in _DTYPE:
            raise ValueError(f"q_out: unsupported dtype {ot}")
        qo, qost = _like(q_out, "q_out", shape, ot, dev)
        ko, kost = (None, 0) if k is None else _like(k_out, "k_out", k.shape, ot, dev)
    code = _call(_abi.load().dsa_idx_norm_rope, dev, (
        *rows, _DTYPE[dt], *wp, wt, _NORM[norm], eps, pos, T, H, Hk, D, R, rope_base, freq, int(rope_interleaved), qo, qost,
        ko, kost, _DTYPE[ot]))
    if code:
        raise _error(code, "dsa_idx_norm_rope")
    return q_out, k_out


def norm_rope_workspace(head_dim: int, device=None) -> torch.Tensor:
    """Device workspace (uint8, 256-byte aligned) for norm_rope_backward."""
    n = _abi.load().dsa_idx_norm_rope_workspace_size(head_dim)
    if n == 0:
        raise ValueError("head_dim must be 64 or 128")
    return torch.empty(n, dtype=torch.uint8, device="cuda" if device is None else device)


def norm_rope_backward(dq_out: torch.Tensor, dk_out: Optional[torch.Tensor], q: torch.Tensor, k: Optional[torch.Tensor],
                       positions: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                       k_weight: Optional[torch.Tensor] = None, norm: str = "rms", eps: float = 1e-6,
                       rope_dim: Optional[int] = None, rope_base: float = 10000.0,
                       inv_freq: Optional[Sequence[float]] = None, rope_interleaved: bool = False,
                       ws: Optional[torch.Tensor] = None) -> NormRopeGrads:
    """Gradients of norm_rope from those of its outputs (dsa_idx_norm_rope_backward).

    q, k, positions and the options as the forward call had them (q and k as
    they were before it); dq_out, dk_out [tokens, heads, head_dim], fp32 or bf16.
    Returns gradients of q and k in their dtype, and in fp32 [head_dim] those of
    the weights (summed over tokens and heads; given or not) and, with norm
    "layer", of the biases."""
    shape, dev, dt, Hk, rows, R, pos, wp, wt, freq = _inputs(q, k, positions, (q_weight, k_weight, None, None), norm, rope_dim,
                                                            inv_freq)
    T, H, D = shape
    gt = dq_out.dtype
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out must both be given or both be None")
    if gt not in _DTYPE:
        raise ValueError(f"dq_out: unsupported dtype {gt}")
    gq, gqst = _like(dq_out, "dq_out", shape, gt, dev)
    gk, gkst = (None, 0) if k is None else _like(dk_out, "dk_out", k.shape, gt, dev)
    dq, dk, dkp = _empty((T, H, D), dt, dev), None, None
    if k is not None:
        dk = _empty((T, Hk, D), dt, dev)
        dkp = dk.data_ptr() or None
    lay = norm == "layer"   # gradients of weights, then of biases, of queries and of keys
    sums = [_empty((D,), torch.float32, dev) if (lay or i < 2) and (k is not None or i % 2 == 0) else None for i in range(4)]
    if ws is None:
        ws = norm_rope_workspace(D, dev)
    code = _call(_abi.load().dsa_idx_norm_rope_backward, dev, (
        gq, gqst, gk, gkst, _DTYPE[gt], *rows, _DTYPE[dt], wp[0], wp[1], wt, _NORM[norm], eps, pos, T, H, Hk, D, R, rope_base,
        freq, int(rope_interleaved), dq.data_ptr() or None, 0, dkp, 0,
        *[None if s is None else s.data_ptr() for s in sums], _arg(ws, "ws", dev, torch.uint8), ws.numel()))
    if code:
        raise _error(code, "dsa_idx_norm_rope_backward")
    return NormRopeGrads(dq, dk, *sums)
