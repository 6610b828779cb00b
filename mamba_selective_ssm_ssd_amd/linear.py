"""torch-facing wrapper of linear attention with a decay for each head
(include/m3_linear.h): ``prefill`` over packed sequences, ``backward`` and
``decode_step``.

    S_t = exp(log_decay) S_{t-1} + k_t v_t^T,      o_t = scale q_t^T S_t

q [T,Hq,Dk], k [T,Hk,Dk], v [T,Hv,Dv] in float32 or bfloat16; each head count
divides H = max(Hq,Hk,Hv), and head h reads row h // (H // Hq) of q (k and v
likewise).  log_decay [H] float32.  Dk and Dv are multiples of 8 up to 128.
Channels of a row must be contiguous and rows 16-byte aligned; the token and
head axes may have any stride that is a multiple of 8 elements, so slices of
one projection's output need no copy.

Sequences are packed along T: ``cu_seqlens`` [B+1] int32 on the device gives
sequence b the tokens cu_seqlens[b]:cu_seqlens[b+1] (empty ones included).
Without it the rows are one sequence, or, given as [B,T,H,D], B sequences of T
tokens.  ``max_seqlen`` (an int) helps to plan; the result does not depend on it
beyond rounding.

States are [n,H,Dk,Dv], float32 or bfloat16.  ``slots`` [B] int32 on the device
names each sequence's state of a pool; a slot outside 0..n-1 marks padding,
whose outputs and state are left as they were; where sequences of one call
share a slot, the first has it and the others' outputs are NaN.

As with ``mixer``, torch only holds memory and names the current stream; all
tensors must be on the current device.
"""
from __future__ import annotations

import torch

from . import capi
from .mixer import _IO, _ptr, _stream


def _flat(t: torch.Tensor, name: str):
    """[T,H,D], or [B,T,H,D] with evenly spaced tokens -> (B or None, T, H, D, token stride, head stride)."""
    if t.dim() == 4:
        b, n, h, d = t.shape
        if b > 1 and n > 1 and h * d > 0 and t.stride(0) != n * t.stride(1):
            raise ValueError(f"{name}: sequences of a [B,T,H,D] tensor must follow each other at the tokens' stride")
        return b, b * n, h, d, t.stride(1) if n > 1 else t.stride(0), t.stride(2)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T,H,D] or [B,T,H,D], got {tuple(t.shape)}")
    return (None, *t.shape, t.stride(0), t.stride(1))


def _rows(t: torch.Tensor, name: str, dtype, device) -> tuple[capi.m3_rows_t, tuple]:
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    b, n, h, d, ts, hs = _flat(t, name)
    if d > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the channels of a row must be contiguous")
    # the stride of an axis of one is of no account, and torch's may be anything
    return capi.m3_rows_t(t.data_ptr(), ts if n > 1 else 0, hs if h > 1 else 0), (b, n, h, d)


def _device(t: torch.Tensor):
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"tensors must be on the current device, got {t.device}")
    return t.device


def _index(t, name: str, n: int | None, device) -> int | None:
    if t is None:
        return None
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dim() != 1 or (n is not None and t.numel() != n):
        raise ValueError(f"{name} must have shape ({n},), got {tuple(t.shape)}")
    return _ptr(t, name, torch.int32)


def _pool(t, name: str, n: int | None, H, dk, dv, device, dtype) -> int | None:
    """Address of a state pool [n,H,Dk,Dv] (any n where None)."""
    if t is None:
        return None
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dim() != 4 or tuple(t.shape[1:]) != (H, dk, dv) or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must be [{'n' if n is None else n},{H},{dk},{dv}], got {tuple(t.shape)}")
    return _ptr(t, name, dtype)


def _decay(t, H, device) -> int:
    if t.device != device or tuple(t.shape) != (H,):
        raise ValueError(f"log_decay must be [{H}] on {device}, got {tuple(t.shape)} on {t.device}")
    return _ptr(t, "log_decay", torch.float32)


def _operands(q, k, v):
    dev, io = _device(q), q.dtype
    if io not in _IO:
        raise ValueError(f"q must be float32 or bfloat16, got {io}")
    (rq, (b, T, hq, dk)), (rk, sk), (rv, sv) = (_rows(t, n, io, dev) for t, n in ((q, "q"), (k, "k"), (v, "v")))
    if sk[:2] != (b, T) or sv[:2] != (b, T) or sk[3] != dk:
        raise ValueError(f"q, k, v must share tokens, and q and k channels: {tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)}")
    return dev, io, (rq, rk, rv), b, T, (hq, sk[2], sv[2]), dk, sv[3]


def make_shape(batch, tokens, q_heads, k_heads, v_heads, key_dim, value_dim, io_dtype=torch.bfloat16,
               state_dtype=torch.float32, max_seqlen=0, scale=1.0) -> capi.m3_linear_shape_t:
    return capi.m3_linear_shape_t(batch, tokens, max_seqlen, q_heads, k_heads, v_heads, key_dim, value_dim,
                                  _IO[io_dtype], _IO[state_dtype], scale)


def _sequences(b, T, cu_seqlens, device):
    """(batch, address of cu_seqlens or None)."""
    if cu_seqlens is None:
        return (1 if b is None else b), None
    if b is not None and b != 1:
        raise ValueError("cu_seqlens needs rows packed along one axis")
    cu = _index(cu_seqlens, "cu_seqlens", None, device)
    if cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must have at least two entries")
    return cu_seqlens.numel() - 1, cu


def _workspace(workspace, need, device, where):
    if need == 0:
        raise capi.M3Error(capi.M3_ERR_UNSUPPORTED, where)
    if workspace is None:
        workspace = torch.empty(need, device=device, dtype=torch.uint8)
    elif workspace.device != device:
        raise ValueError(f"workspace must be on {device}, got {workspace.device}")
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def workspace_bytes(q, k, v, cu_seqlens=None, max_seqlen=0, backward=False) -> int:
    """Bytes of the workspace that ``prefill`` (or ``backward``) takes for these operands."""
    dev, io, _, b, T, heads, dk, dv = _operands(q, k, v)
    batch, _ = _sequences(b, T, cu_seqlens, dev)
    shape = make_shape(batch, T, *heads, dk, dv, io, max_seqlen=max_seqlen or 0)
    return (capi.m3_linear_prefill_backward_workspace_bytes if backward
            else capi.m3_linear_prefill_workspace_bytes)(shape)


def prefill(q, k, v, log_decay, state=None, final=None, want_final=True, *, cu_seqlens=None, max_seqlen=None,
            slots=None, scale=None, o=None, workspace=None, state_dtype=None):
    """Prompt pass.  Returns (o, final): o [T,H,Dv] ([B,T,H,Dv] for such rows).

    ``state`` holds the states to start from (None: zeros).  The states behind
    the last tokens go to ``final`` if given, else to ``state`` (in place) when
    one was given, else to new ones in sequence order (``state_dtype``, default
    float32) -- unless want_final=False.  With ``slots``, ``state`` and
    ``final`` are pools of one size, and one of them must be given unless
    want_final=False.  ``scale`` defaults to Dk ** -0.5.
    """
    dev, io, rows, b, T, heads, dk, dv = _operands(q, k, v)
    H = max(heads)
    batch, cu = _sequences(b, T, cu_seqlens, dev)
    given = state if state is not None else final
    sd = given.dtype if given is not None else (state_dtype or torch.float32)
    if sd not in _IO or (state_dtype is not None and state_dtype != sd) or (final is not None and final.dtype != sd):
        raise ValueError("initial and final states must share one state dtype, float32 or bfloat16")
    if not want_final:
        final = None
    elif final is None:
        if state is None and slots is not None:
            raise ValueError("slots need a state pool: give final, or want_final=False")
        final = state if state is not None else torch.empty(batch, H, dk, dv, device=dev, dtype=sd)
    n = batch if slots is None else (state if state is not None else final).shape[0] if (state is not None or final is not None) else batch
    shape = capi.m3_linear_shape_t(batch, T, max_seqlen or 0, *heads, dk, dv, _IO[io], _IO[sd],
                                   dk ** -0.5 if scale is None else scale)
    out_shape = (T, H, dv) if b is None else (b, T // b if b else 0, H, dv)
    if o is None:
        o = torch.empty(out_shape, device=dev, dtype=io)
    elif tuple(o.shape) != out_shape:
        raise ValueError(f"o must be {out_shape}, got {tuple(o.shape)}")
    workspace, wp, wn = _workspace(workspace, capi.m3_linear_prefill_workspace_bytes(shape), dev, "m3_linear_prefill")
    rc = capi.m3_linear_prefill(shape, *rows, _decay(log_decay, H, dev), cu, _index(slots, "slots", batch, dev), n,
                                _pool(state, "state", n, H, dk, dv, dev, sd),
                                _pool(final, "final", n, H, dk, dv, dev, sd), _rows(o, "o", io, dev)[0], wp, wn,
                                _stream())
    if rc != capi.M3_OK:
        raise capi.M3Error(rc, "m3_linear_prefill")
    return o, final


def decode_step(q, k, v, log_decay, state, *, slots=None, scale=None, o=None):
    """One token of every sequence: q [B,Hq,Dk], k [B,Hk,Dk], v [B,Hv,Dv].
    Updates ``state`` [n,H,Dk,Dv] (row b, or row slots[b]) in place and returns
    o [B,H,Dv]."""
    dev, io, rows, b, B, heads, dk, dv = _operands(q, k, v)
    if b is not None:
        raise ValueError("decode_step takes rows [B,H,D]")
    H = max(heads)
    if B == 0:
        raise capi.M3Error(capi.M3_ERR_INVALID_ARGUMENT, "m3_linear_decode_step")
    if state.dtype not in _IO:
        raise ValueError(f"state must be float32 or bfloat16, got {state.dtype}")
    if o is None:
        o = torch.empty(B, H, dv, device=dev, dtype=io)
    elif tuple(o.shape) != (B, H, dv):
        raise ValueError(f"o must be {(B, H, dv)}, got {tuple(o.shape)}")
    shape = capi.m3_linear_shape_t(B, B, 0, *heads, dk, dv, _IO[io], _IO[state.dtype], dk ** -0.5 if scale is None else scale)
    rc = capi.m3_linear_decode_step(shape, *rows, _decay(log_decay, H, dev), _index(slots, "slots", B, dev),
                                    state.shape[0],
                                    _pool(state, "state", None if slots is not None else B, H, dk, dv, dev, state.dtype),
                                    _rows(o, "o", io, dev)[0], _stream())
    if rc != capi.M3_OK:
        raise capi.M3Error(rc, "m3_linear_decode_step")
    return o


def backward(q, k, v, log_decay, go, state=None, gfinal=None, *, cu_seqlens=None, max_seqlen=None, scale=None,
             workspace=None):
    """Gradients of sum(go * o) + <gfinal, final> for o, final = prefill(q, ...,
    state=state).  Returns a dict of q, k and v, shaped and typed like the
    inputs, and, when ``state`` [B,H,Dk,Dv] is given, state (float32).
    ``gfinal`` [B,H,Dk,Dv] float32 or None.  log_decay has no gradient: it is a
    constant of the layer."""
    dev, io, rows, b, T, heads, dk, dv = _operands(q, k, v)
    H = max(heads)
    batch, cu = _sequences(b, T, cu_seqlens, dev)
    rg, sg = _rows(go, "go", io, dev)
    if sg != (b, T, H, dv):
        raise ValueError(f"go must be shaped like o, got {tuple(go.shape)}")
    sd = state.dtype if state is not None else torch.float32
    if sd not in _IO:
        raise ValueError(f"state must be float32 or bfloat16, got {sd}")
    shape = capi.m3_linear_shape_t(batch, T, max_seqlen or 0, *heads, dk, dv, _IO[io], _IO[sd],
                                   dk ** -0.5 if scale is None else scale)
    g = {n: torch.empty(t.shape, device=dev, dtype=io) for n, t in (("q", q), ("k", k), ("v", v))}
    if state is not None:
        g["state"] = torch.empty(batch, H, dk, dv, device=dev, dtype=torch.float32)
    workspace, wp, wn = _workspace(workspace, capi.m3_linear_prefill_backward_workspace_bytes(shape), dev,
                                   "m3_linear_prefill_backward")
    rc = capi.m3_linear_prefill_backward(
        shape, *rows, _decay(log_decay, H, dev), cu, _pool(state, "state", batch, H, dk, dv, dev, sd), rg,
        _pool(gfinal, "gfinal", batch, H, dk, dv, dev, torch.float32), *(_rows(g[n], n, io, dev)[0] for n in "qkv"),
        g["state"].data_ptr() if state is not None else None, wp, wn, _stream())
    if rc != capi.M3_OK:
        raise capi.M3Error(rc, "m3_linear_prefill_backward")
    return g
