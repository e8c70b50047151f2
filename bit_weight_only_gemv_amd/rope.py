"""Norm and rotation of queries and keys (include/wq.h, "norm and rotation of
queries and keys"), between a projection and the key/value caches:

    q, k = wq_qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, 1e-6)
"""

from __future__ import annotations

import ctypes

from . import _lib as L
from .kv4 import _dtype, _new, _strided
from .kv8 import _same_device


_NONE = L.Heads(None, None, None, 0, 0, 0, 0, 0)


def _side(x, weight, out, stream, what):
    """wq_heads of one of the two, and its result."""
    if x is None:
        if weight is not None or out is not None:
            raise ValueError(f"{what} is missing, but not its weight or output")
        return _NONE, None
    p, r, h = _strided(x, what)
    if out is None:
        out = _new(x.shape, x.dtype, x.device, stream)
    elif out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError(f"{what}'s output must have its shape and type")
    op, orow, ohead = _strided(out, what)
    wp = None
    if weight is not None:
        if weight.shape != x.shape[2:] or weight.dtype != x.dtype:
            raise ValueError(f"{what}'s weight must be [{x.shape[2]}] of its type")
        wp = L._dptr(weight)
        _same_device(x, out, weight)
    else:
        _same_device(x, out)
    return L.Heads(p, op, wp, x.shape[1], r, h, orow, ohead), out


def wq_qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, q_out=None,
                    k_out=None, neighbours=False, stream=None):
    """Divides every head of q [rows, heads, D] and k [rows, kv_heads, D] by its root
    mean square (eps None: not), weights it with q_weight or k_weight [D], and rotates
    its first 2 n channels by positions int32 [rows] times inv_freq float64 [n]: pairs
    (j, n + j), with `neighbours` (2 j, 2 j + 1).  inv_freq None: no rotation.  q or k
    may be None, outputs their inputs (in place).  Returns both outputs."""
    import torch
    fn = L.load().wq_qk_norm_rope
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k is needed")
    rows, _, channels = x.shape
    if q is not None and k is not None and (rows != k.shape[0] or channels != k.shape[2] or q.dtype != k.dtype):
        raise ValueError("q and k must have the same rows, channels and type")
    if eps is None:
        if q_weight is not None or k_weight is not None:
            raise ValueError("weights belong to the norm: eps is None")
        eps = -1.0
    elif not eps >= 0:
        raise ValueError(f"eps must be at least 0, got {eps}")
    a, q_out = _side(q, q_weight, q_out, stream, "q")
    b, k_out = _side(k, k_weight, k_out, stream, "k")
    n, pp, fp = 0, None, None
    if inv_freq is not None:
        n = inv_freq.numel()
        if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be float64 [n]")
        if positions is None:
            raise ValueError("inv_freq needs positions")
        pp, fp = L._i32(positions, (rows,), "positions"), L._dptr(inv_freq)
        _same_device(positions, inv_freq)
    L._check(fn(_dtype(x), ctypes.addressof(a), ctypes.addressof(b), rows, channels, eps, pp, fp, n,
                bool(neighbours), L._stream(stream)))
    return q_out, k_out
