"""torch-facing wrapper of linear attention with a decay for each head
(include/m3_linear.h): ``prefill`` over packed sequences, ``backward`` and
``decode_step``.

    S_t = exp(log_decay) S_{t-1} + k_t v_t^T,      o_t = scale q_t^T S_t

q [T,Hq,Dk], k [T,Hk,Dk], v [T,Hv,Dv] in float32 or bfloat16; each head count
divides H = max(Hq,Hk,Hv), and head h reads row h // (H // Hq) of q (k and v
likewise).  log_decay [H] float32.  Dk and Dv are multiples of 8 up to 128.
Channels of a row must be contiguous and rows 16-byte aligned; the token and
head axes may have any stride that is a multiple of 8 elements, the tokens' at
least a row's channels, so slices of one projection's output need no copy.

Sequences are packed along T: ``cu_seqlens`` [B+1] int32 on the device gives
sequence b the tokens cu_seqlens[b]:cu_seqlens[b+1] (empty ones included).
Without it the rows are one sequence, or, given as [B,T,H,D], B sequences of T
tokens.  Rows outside every sequence are not read, and their rows of o not
written (undefined in a new one); their gradients are zero.  ``max_seqlen``
(an int) helps to plan; the result does not depend on it beyond rounding.  Give
it where sequences are many: without it one of them may be all of T, and enough
of them to fill the chip are cut into segments all the same, with a workspace of
an fp32 state per segment and head, and k and v read twice.

States are [n,H,Dk,Dv], float32 or bfloat16.  ``slots`` [B] int32 on the device
names each sequence's state of a pool; a slot outside 0..n-1 (without a pool: a
negative one) marks padding, whose outputs and state are left as they were;
where sequences of one call share a slot, the first has it and the others'
outputs are NaN.

As with ``mixer``, torch only holds memory and names the current stream; all
tensors must be on the current device.
"""
from __future__ import annotations

import torch

from . import capi
from .mixer import _IO


# A step of a few rows is over in the time that its wrapper takes, so the checks
# read each tensor's shape and strides once and compare devices by number.

def _stream(device: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device)   # current_stream() without its object


def _device(t: torch.Tensor) -> int:
    device = t.get_device()
    if device < 0 or device != torch.cuda.current_device():
        raise ValueError(f"tensors must be on the current device, got {t.device}")
    return device


def _rows(t: torch.Tensor, name: str, dtype, device: int):
    """(rows, (B or None, tokens, heads, channels)) of [T,H,D], or of [B,T,H,D] with evenly spaced tokens."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        b, (n, h, d), (ts, hs, cs) = None, shape, stride
    elif len(shape) == 4:
        (b, n, h, d), (bs, ts, hs, cs) = shape, stride
        if n == 1:
            ts = bs
        elif b > 1 and h * d > 0 and bs != n * ts:
            raise ValueError(f"{name}: sequences of a [B,T,H,D] tensor must follow each other at the tokens' stride")
        n *= b
    else:
        raise ValueError(f"{name} must be [T,H,D] or [B,T,H,D], got {tuple(shape)}")
    if cs != 1 and d > 1:
        raise ValueError(f"{name}: the channels of a row must be contiguous")
    # the stride of an axis of one is of no account, and torch's may be anything
    return capi.m3_rows_t(t.data_ptr(), ts if n > 1 else 0, hs if h > 1 else 0), (b, n, h, d)


def _like_rows(t: torch.Tensor, heads: int, channels: int):
    """A new contiguous tensor of the shape and type of rows ``t``, and its rows."""
    new = torch.empty_like(t, memory_format=torch.contiguous_format)
    return new, capi.m3_rows_t(new.data_ptr(), heads * channels, channels)


def _ptr(t, name: str, shape: tuple | None, dtype, device: int) -> int | None:
    """Address of a contiguous tensor of that shape and type (None for None)."""
    if t is None:
        return None
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _operands(q, k, v):
    """device, I/O type and its number, rows, B or None, tokens, head counts, Dk, Dv."""
    dev, io = _device(q), q.dtype
    ion = _IO.get(io)
    if ion is None:
        raise ValueError(f"q must be float32 or bfloat16, got {io}")
    rq, (b, T, hq, dk) = _rows(q, "q", io, dev)
    rk, (bk, Tk, hk, dkk) = _rows(k, "k", io, dev)
    rv, (bv, Tv, hv, dv) = _rows(v, "v", io, dev)
    if bk != b or bv != b or Tk != T or Tv != T or dkk != dk:
        raise ValueError(f"q, k, v must share tokens, and q and k channels: {tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)}")
    return dev, io, ion, rq, rk, rv, b, T, (hq, hk, hv), dk, dv


def make_shape(batch, tokens, q_heads, k_heads, v_heads, key_dim, value_dim, io_dtype=torch.bfloat16,
               state_dtype=torch.float32, max_seqlen=0, scale=1.0) -> capi.m3_linear_shape_t:
    return capi.m3_linear_shape_t(batch, tokens, max_seqlen, q_heads, k_heads, v_heads, key_dim, value_dim,
                                  _IO[io_dtype], _IO[state_dtype], scale)


def _sequences(b, T, cu_seqlens, device: int):
    """(batch, address of cu_seqlens or None, longest sequence that may be)."""
    if cu_seqlens is None:
        return (1, None, T) if b is None else (b, None, T // b if b else 0)
    if b is not None and b != 1:
        raise ValueError("cu_seqlens needs rows packed along one axis")
    cu = _ptr(cu_seqlens, "cu_seqlens", None, torch.int32, device)
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError(f"cu_seqlens must be [B+1] with two entries or more, got {tuple(cu_seqlens.shape)}")
    return cu_seqlens.shape[0] - 1, cu, T


def _workspace(workspace, need: int, like: torch.Tensor, device: int, where: str):
    """(address, bytes, owner) of the given workspace or a new one."""
    if workspace is None:
        if need == 0:
            raise capi.M3Error(capi.M3_ERR_UNSUPPORTED, where)
        workspace = like.new_empty((need,), dtype=torch.uint8)
        return workspace.data_ptr(), need, workspace
    if workspace.get_device() != device:
        raise ValueError(f"workspace must be on cuda:{device}, got {workspace.device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def workspace_bytes(q, k, v, cu_seqlens=None, max_seqlen=0, backward=False) -> int:
    """Bytes of the workspace that ``prefill`` (or ``backward``) takes for these
    operands, and the same max_seqlen."""
    dev, io, ion, _, _, _, b, T, heads, dk, dv = _operands(q, k, v)
    batch, _, longest = _sequences(b, T, cu_seqlens, dev)
    shape = make_shape(batch, T, *heads, dk, dv, io, max_seqlen=max_seqlen or longest)
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
    dev, io, ion, rq, rk, rv, b, T, heads, dk, dv = _operands(q, k, v)
    H = max(heads)
    batch, cu, longest = _sequences(b, T, cu_seqlens, dev)
    given = state if state is not None else final
    sd = given.dtype if given is not None else (state_dtype or torch.float32)
    if sd not in _IO or (state_dtype is not None and state_dtype != sd) or (final is not None and final.dtype != sd):
        raise ValueError("initial and final states must share one state dtype, float32 or bfloat16")
    if not want_final:
        final = None
    elif final is None:
        if state is None and slots is not None:
            raise ValueError("slots need a state pool: give final, or want_final=False")
        final = state if state is not None else torch.empty((batch, H, dk, dv), device=q.device, dtype=sd)
    # without a pool any slot from 0 on is one of its own
    n = batch if slots is None else given.shape[0] if given is not None else 1 << 31
    shape = capi.m3_linear_shape_t(batch, T, max_seqlen or longest, *heads, dk, dv, ion, _IO[sd],
                                   dk ** -0.5 if scale is None else scale)
    out_shape = (T, H, dv) if b is None else (b, T // b if b else 0, H, dv)
    if o is None:
        o = q.new_empty(out_shape)
        ro = capi.m3_rows_t(o.data_ptr(), H * dv, dv)
    elif o.shape != out_shape:
        raise ValueError(f"o must be {out_shape}, got {tuple(o.shape)}")
    else:
        ro, _ = _rows(o, "o", io, dev)
    wp, wn, workspace = _workspace(workspace, capi.m3_linear_prefill_workspace_bytes(shape), q, dev,
                                   "m3_linear_prefill")
    pool = (n, H, dk, dv)
    rc = capi.m3_linear_prefill(shape, rq, rk, rv, _ptr(log_decay, "log_decay", (H,), torch.float32, dev), cu,
                                _ptr(slots, "slots", (batch,), torch.int32, dev), n, _ptr(state, "state", pool, sd, dev),
                                _ptr(final, "final", pool, sd, dev), ro, wp, wn, _stream(dev))
    if rc:
        raise capi.M3Error(rc, "m3_linear_prefill")
    return o, final


def decode_step(q, k, v, log_decay, state, *, slots=None, scale=None, o=None):
    """One token of every sequence: q [B,Hq,Dk], k [B,Hk,Dk], v [B,Hv,Dv].
    Updates ``state`` [n,H,Dk,Dv] (row b, or row slots[b]) in place and returns
    o [B,H,Dv]."""
    dev, io, ion, rq, rk, rv, b, B, heads, dk, dv = _operands(q, k, v)
    if b is not None:
        raise ValueError("decode_step takes rows [B,H,D]")
    H = max(heads)
    if B == 0:
        raise capi.M3Error(capi.M3_ERR_INVALID_ARGUMENT, "m3_linear_decode_step")
    sd = state.dtype
    if sd not in _IO:
        raise ValueError(f"state must be float32 or bfloat16, got {sd}")
    if o is None:
        o = q.new_empty((B, H, dv))
        ro = capi.m3_rows_t(o.data_ptr(), H * dv, dv)
    elif o.shape != (B, H, dv):
        raise ValueError(f"o must be {(B, H, dv)}, got {tuple(o.shape)}")
    else:
        ro, _ = _rows(o, "o", io, dev)
    n = B if slots is None else state.shape[0]
    shape = capi.m3_linear_shape_t(B, B, 0, *heads, dk, dv, ion, _IO[sd], dk ** -0.5 if scale is None else scale)
    rc = capi.m3_linear_decode_step(shape, rq, rk, rv, _ptr(log_decay, "log_decay", (H,), torch.float32, dev),
                                    _ptr(slots, "slots", (B,), torch.int32, dev), n,
                                    _ptr(state, "state", (n, H, dk, dv), sd, dev), ro, _stream(dev))
    if rc:
        raise capi.M3Error(rc, "m3_linear_decode_step")
    return o


def backward(q, k, v, log_decay, go, state=None, gfinal=None, *, cu_seqlens=None, max_seqlen=None, scale=None,
             workspace=None):
    """Gradients of sum(go * o) + <gfinal, final> for o, final = prefill(q, ...,
    state=state).  Returns a dict of q, k and v, shaped and typed like the
    inputs, and, when ``state`` [B,H,Dk,Dv] is given, state (float32).
    ``gfinal`` [B,H,Dk,Dv] float32 or None.  log_decay has no gradient: it is a
    constant of the layer."""
    dev, io, ion, rq, rk, rv, b, T, heads, dk, dv = _operands(q, k, v)
    H = max(heads)
    batch, cu, longest = _sequences(b, T, cu_seqlens, dev)
    rg, sg = _rows(go, "go", io, dev)
    if sg != (b, T, H, dv):
        raise ValueError(f"go must be shaped like o, got {tuple(go.shape)}")
    sd = state.dtype if state is not None else torch.float32
    if sd not in _IO:
        raise ValueError(f"state must be float32 or bfloat16, got {sd}")
    shape = capi.m3_linear_shape_t(batch, T, max_seqlen or longest, *heads, dk, dv, ion, _IO[sd],
                                   dk ** -0.5 if scale is None else scale)
    (gq, rgq), (gk, rgk), (gv, rgv) = _like_rows(q, heads[0], dk), _like_rows(k, heads[1], dk), _like_rows(v, heads[2], dv)
    g = {"q": gq, "k": gk, "v": gv}
    pool = (batch, H, dk, dv)
    if state is not None:
        g["state"] = torch.empty(pool, device=q.device, dtype=torch.float32)
    wp, wn, workspace = _workspace(workspace, capi.m3_linear_prefill_backward_workspace_bytes(shape), q, dev,
                                   "m3_linear_prefill_backward")
    rc = capi.m3_linear_prefill_backward(
        shape, rq, rk, rv, _ptr(log_decay, "log_decay", (H,), torch.float32, dev), cu,
        _ptr(state, "state", pool, sd, dev), rg, _ptr(gfinal, "gfinal", pool, torch.float32, dev), rgq, rgk, rgv,
        g["state"].data_ptr() if state is not None else None, wp, wn, _stream(dev))
    if rc:
        raise capi.M3Error(rc, "m3_linear_prefill_backward")
    return g
