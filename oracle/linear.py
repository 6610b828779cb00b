"""fp64 oracle of linear attention with a decay for each head and of the norm
with position rotation: token by token, head by head, straight from the
definitions in include/m3_linear.h and include/m3_rotary.h.  Test
infrastructure; shares nothing with the HIP library.
"""
from __future__ import annotations

import numpy as np


def _expand(x, H):
    return np.repeat(x, H // x.shape[1], axis=1)


def _spans(cu):
    return [(int(cu[i]), int(cu[i + 1])) for i in range(len(cu) - 1)]


def prefill(q, k, v, log_decay, cu, state=None, scale=None):
    """q [T,Hq,Dk], k [T,Hk,Dk], v [T,Hv,Dv], state [B,H,Dk,Dv] or None -> (o [T,H,Dv], final)."""
    H = len(log_decay)
    scale = q.shape[2] ** -0.5 if scale is None else scale
    q, k, v = (_expand(np.asarray(x, np.float64), H) for x in (q, k, v))
    g = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    o = np.zeros((q.shape[0], H, v.shape[2]))
    final = np.zeros((len(cu) - 1, H, q.shape[2], v.shape[2])) if state is None else np.array(state, np.float64)
    for b, (lo, hi) in enumerate(_spans(cu)):
        S = final[b]
        for t in range(lo, hi):
            S = g * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hk,hkv->hv", q[t], S)
        final[b] = S
    return o, final


def backward(q, k, v, log_decay, go, cu, state=None, gfinal=None, scale=None):
    """Gradients of sum(go * o) + <gfinal, final>: (dq, dk, dv, dstate)."""
    H = len(log_decay)
    scale = q.shape[2] ** -0.5 if scale is None else scale
    heads = [x.shape[1] for x in (q, k, v)]
    q, k, v = (_expand(np.asarray(x, np.float64), H) for x in (q, k, v))
    go = np.asarray(go, np.float64)
    g = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    shape = (len(cu) - 1, H, q.shape[2], v.shape[2])
    S0 = np.zeros(shape) if state is None else np.asarray(state, np.float64)
    G0 = np.zeros(shape) if gfinal is None else np.array(gfinal, np.float64)
    for b, (lo, hi) in enumerate(_spans(cu)):
        S = S0[b]
        for t in range(lo, hi):
            S = g * S + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * np.einsum("hkv,hv->hk", S, go[t])
        G = G0[b]                                   # dL/dS behind token t
        for t in range(hi - 1, lo - 1, -1):
            G = G + scale * q[t][:, :, None] * go[t][:, None, :]
            dk[t] = np.einsum("hkv,hv->hk", G, v[t])
            dv[t] = np.einsum("hk,hkv->hv", k[t], G)
            G = g * G
        G0[b] = G
    grads = [d.reshape(d.shape[0], n, H // n, d.shape[2]).sum(2) for d, n in zip((dq, dk, dv), heads)]
    return (*grads, G0)


def norm_rotate(x, positions, inv_freq, weight=None, norm=True, eps=1e-6, halves=False):
    """x [T,H,D], positions [axes,T], inv_freq [axes,n] -> turned rows [T,H,D]."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    if norm:
        y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
        if weight is not None:
            y = y * np.asarray(weight, np.float64)
    # in long double: a far position's angle has more whole turns than fp64 leaves bits for
    angle = np.sum(np.asarray(positions, np.longdouble)[:, :, None] * np.asarray(inv_freq, np.longdouble)[:, None], axis=0)
    angle = np.remainder(angle, 8 * np.arctan(np.longdouble(1))).astype(np.float64)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    n = angle.shape[1]
    a, b = (slice(0, n), slice(n, 2 * n)) if halves else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    out = y.copy()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., a] * s + y[..., b] * c
    return out


def norm_rotate_backward(x, positions, inv_freq, g, weight=None, norm=True, eps=1e-6, halves=False):
    """Gradients of sum(g * norm_rotate(x)): (dx, dweight or None)."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    gn = norm_rotate(g, -np.asarray(positions, np.float64), inv_freq, None, False, eps, halves)
    if not norm:
        return gn, None
    w = np.ones(x.shape[-1]) if weight is None else np.asarray(weight, np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    dx = r * w * gn - r ** 3 * x * np.mean(x * w * gn, axis=-1, keepdims=True)
    return dx, None if weight is None else np.sum(gn * x * r, axis=(0, 1))
