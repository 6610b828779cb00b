"""torch-facing wrapper of the norm of queries and keys for each head with the
position rotation in the same pass (include/m3_rotary.h).

    n = w x / sqrt(mean(x^2) + eps),    y = R(angle) n,
    angle_i = sum_a positions[a, token] inv_freq[a, i]

q [T,Hq,D], k [T,Hk,D] (or [B,T,H,D]) in float32 or bfloat16, strided as in
``linear``; positions [T] or [axes,T], int32 or int64; inv_freq [n] or
[axes,n] float32, which turns the first 2 n channels: the pairs (2i, 2i+1), or
(i, i+n) with halves=True.  ``axes_table`` lays out the frequencies of several
axes (time, height, width).  D and 2 n are multiples of 8, D up to 256;
inv_freq and the weights are contiguous and start at multiples of 16 bytes.
"""
from __future__ import annotations

import torch

from . import capi
from .linear import _device, _like_rows, _ptr, _rows, _stream, _workspace
from .mixer import _IO


def axes_table(inv_freq: torch.Tensor, sections, interleaved: bool = False) -> torch.Tensor:
    """[axes,n] frequencies: pair i turns by the position of its axis.

    ``sections`` gives each axis its number of pairs (their sum is n): runs of
    pairs in the axes' order, or, ``interleaved``, dealt out in turn until an
    axis has all of its own.
    """
    n = inv_freq.numel()
    if inv_freq.dim() != 1 or sum(sections) != n or any(s < 0 for s in sections):
        raise ValueError(f"sections must add up to {n} pairs, got {tuple(sections)}")
    if interleaved:
        left, axis = list(sections), []
        while len(axis) < n:
            for a, s in enumerate(left):
                if s > 0:
                    axis.append(a)
                    left[a] -= 1
    else:
        axis = [a for a, s in enumerate(sections) for _ in range(s)]
    pick = torch.tensor(axis, device=inv_freq.device) == torch.arange(len(sections), device=inv_freq.device)[:, None]
    return torch.where(pick, inv_freq, torch.zeros_like(inv_freq)).float().contiguous()


def _out(out, name, x, heads, d, device):
    if out is None:
        return _like_rows(x, heads, d)
    if out.shape != x.shape:
        raise ValueError("q_out and k_out must be shaped like q and k")
    return out, _rows(out, name, x.dtype, device)[0]


def _common(q, k, positions, inv_freq, norm, eps, halves):
    dev, io = _device(q), q.dtype
    if io not in _IO:
        raise ValueError(f"q must be float32 or bfloat16, got {io}")
    rq, (b, T, hq, d) = _rows(q, "q", io, dev)
    rk, (bk, Tk, hk, dk) = _rows(k, "k", io, dev)
    if bk != b or Tk != T or dk != d:
        raise ValueError(f"q and k must share tokens and channels: {tuple(q.shape)}, {tuple(k.shape)}")
    f, pd = inv_freq.shape, positions.dtype
    if len(f) not in (1, 2):
        raise ValueError(f"inv_freq must be [n] or [axes,n], got {tuple(f)}")
    axes = 1 if len(f) == 1 else f[0]
    if pd is not torch.int32 and pd is not torch.int64:
        raise ValueError(f"positions must be int32 or int64, got {pd}")
    if positions.numel() != axes * T or (axes > 1 and positions.shape[0] != axes):
        raise ValueError(f"positions must be [{axes},{T}], got {tuple(positions.shape)}")
    shape = capi.m3_rotary_shape_t(T, hq, hk, d, 2 * f[-1], axes, _IO[io], pd is torch.int64, bool(halves), bool(norm), eps)
    return (dev, io, shape, rq, rk, _ptr(positions, "positions", None, pd, dev),
            _ptr(inv_freq, "inv_freq", None, torch.float32, dev), hq, hk, d)


def norm_rotate(q, k, positions, inv_freq, *, norm=True, eps=1e-6, q_weight=None, k_weight=None, halves=False,
                q_out=None, k_out=None):
    """Returns (q', k'), shaped like q and k (new ones, or ``q_out`` and
    ``k_out``, which may be q and k themselves).  ``q_weight`` and ``k_weight``
    [D] float32 belong to the norm; norm=False only turns."""
    dev, io, shape, rq, rk, pos, freq, hq, hk, d = _common(q, k, positions, inv_freq, norm, eps, halves)
    q_out, ro = _out(q_out, "q_out", q, hq, d, dev)
    k_out, rko = _out(k_out, "k_out", k, hk, d, dev)
    rc = capi.m3_norm_rotate(shape, rq, rk, pos, freq, _ptr(q_weight, "q_weight", (d,), torch.float32, dev),
                             _ptr(k_weight, "k_weight", (d,), torch.float32, dev), ro, rko, _stream(dev))
    if rc:
        raise capi.M3Error(rc, "m3_norm_rotate")
    return q_out, k_out


def norm_rotate_backward(q, k, positions, inv_freq, gq, gk, *, norm=True, eps=1e-6, q_weight=None, k_weight=None,
                         halves=False, workspace=None):
    """Gradients of sum(gq * q') + sum(gk * k') for q', k' = norm_rotate(q, k,
    ...): a dict of q and k, and q_weight and k_weight (float32) where given."""
    dev, io, shape, rq, rk, pos, freq, hq, hk, d = _common(q, k, positions, inv_freq, norm, eps, halves)
    if gq.shape != q.shape or gk.shape != k.shape:
        raise ValueError("gq and gk must be shaped like q and k")
    wp, wn, workspace = _workspace(workspace, capi.m3_norm_rotate_backward_workspace_bytes(shape), q, dev,
                                   "m3_norm_rotate_backward")
    pqw, pkw = _ptr(q_weight, "q_weight", (d,), torch.float32, dev), _ptr(k_weight, "k_weight", (d,), torch.float32, dev)
    (dq, rdq), (dk, rdk) = _like_rows(q, hq, d), _like_rows(k, hk, d)
    g, pdq, pdk = {"q": dq, "k": dk}, None, None
    if q_weight is not None:
        g["q_weight"] = torch.empty_like(q_weight)
        pdq = g["q_weight"].data_ptr()
    if k_weight is not None:
        g["k_weight"] = torch.empty_like(k_weight)
        pdk = g["k_weight"].data_ptr()
    rc = capi.m3_norm_rotate_backward(shape, rq, rk, pos, freq, pqw, pkw, _rows(gq, "gq", io, dev)[0],
                                      _rows(gk, "gk", io, dev)[0], rdq, rdk, pdq, pdk, wp, wn, _stream(dev))
    if rc:
        raise capi.M3Error(rc, "m3_norm_rotate_backward")
    return g
