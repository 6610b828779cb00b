"""Workloads of the linear-attention and rotary operators, with plain forms to compare against.

Every case makes one call of ``linear.prefill``, ``linear.backward``,
``linear.decode_step``, ``rotary.norm_rotate`` or
``rotary.norm_rotate_backward``.  ``run`` computes it with elementary torch
operations, or through the package where ``own`` is set; ``exact`` gives the
same outputs in 64 bits from the token-by-token definition.

    S_t = exp(log_decay) S_{t-1} + k_t v_t^T,      o_t = scale q_t^T S_t
    y = R(angle) (w x / sqrt(mean x^2 + eps)),     angle_i = sum_a position_a inv_freq[a, i]
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_CHUNK = 64


# ---- the cases -------------------------------------------------------------

def _prefill(name, dtype, batch, tokens, heads, dk, dv, **kw):
    c = dict(name=name, op="prefill", dtype=dtype, batch=batch, tokens=tokens, q_heads=heads, k_heads=heads,
             v_heads=heads, dk=dk, dv=dv, ragged=True, state=False, fused=False)
    c.update(kw)
    return c


def _rotary(name, op, dtype, tokens, q_heads, k_heads, dim, rot, **kw):
    c = dict(name=name, op=op, dtype=dtype, tokens=tokens, q_heads=q_heads, k_heads=k_heads, dim=dim, rot=rot,
             axes=1, halves=True, norm=True, weight=True, far=False, fused=False)
    c.update(kw)
    return c


def listed():
    return [
        # sixteen prompts of different lengths in one call, as a server admits them: lengths of 0 and 1 among them
        _prefill("prefill_packed", "bf16", 16, 16384, 32, 128, 128),
        # one long context at the mixer's own long workload: 65536 tokens, 64 heads of 64
        _prefill("prefill_long", "bf16", 1, 65536, 64, 64, 64, ragged=False),
        # the next piece of one prompt from a carried state, grouped k and v heads: latency counts
        _prefill("prefill_piece", "bf16", 1, 77, 16, 128, 128, k_heads=4, v_heads=4, state=True),
        # full-precision evaluation of two sequences, key and value sizes that differ
        _prefill("prefill_f32", "f32", 2, 4096, 16, 64, 128, ragged=False, state=True),
        # the training batch of the mixer's own workloads: 4 x 2048 tokens, 64 heads of 64
        _prefill("backward_train", "bf16", 4, 8192, 64, 64, 64, op="backward", ragged=False),
        # packed documents with grouped heads and carried states (truncated backpropagation)
        _prefill("backward_grouped", "bf16", 7, 4999, 32, 128, 128, op="backward", k_heads=8, v_heads=8, state=True),
        # one token of 256 requests, 64 heads of 64: the mixer's own decode batch
        _prefill("decode_batch", "bf16", 256, 256, 64, 64, 64, op="decode", pool=256, state_dtype="f32"),
        # one token of three requests somewhere in a pool of states: latency counts
        _prefill("decode_few", "bf16", 3, 3, 32, 128, 128, op="decode", pool=9, state_dtype="f32", k_heads=8, v_heads=8),
        # queries and keys of a packed prompt, views of one projection's rows
        _rotary("rotary_prompt", "rotary", "bf16", 16384, 32, 8, 128, 128, fused=True),
        # one token each of five requests far into their contexts
        _rotary("rotary_step", "rotary", "bf16", 5, 16, 16, 64, 32, halves=False, far=True),
        # the training batch's gradients, adjacent pairs
        _rotary("rotary_backward_train", "rotary_backward", "bf16", 8192, 64, 64, 64, 64, halves=False),
        # gradients for image and video positions (time, height, width) in full precision
        _rotary("rotary_backward_axes", "rotary_backward", "f32", 3001, 16, 4, 96, 96, axes=3),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_heads(rng, most):
    heads = rng.choice([h for h in (1, 2, 3, 5, 6, 8, 12, 16, 24, 32, 40, 64) if h <= most])
    shared = rng.choice([d for d in (1, 2, 3, 4, 8) if heads % d == 0])
    kind = rng.randrange(3)  # all heads alike; grouped k and v; shared q and k under more values
    return {0: (heads, heads, heads), 1: (heads, heads // shared, heads // shared),
            2: (heads // shared, heads // shared, heads)}[kind]


def _draw_scan(rng, op):
    dk, dv = rng.choice((16, 32, 48, 64, 80, 96, 128)), rng.choice((16, 32, 64, 64, 96, 112, 128))
    qh, kh, vh = _draw_heads(rng, 64)
    dtype = rng.choice(("bf16", "bf16", "f32"))
    # elements of o at most those of the largest listed case of the direction
    most = {"prefill": 1 << 26, "backward": 1 << 24}[op]
    most = min(1 << 16, most // (max(qh, kh, vh) * max(dk, dv))) // (4 if dtype == "f32" else 1)
    tokens = _log_int(rng, 1, max(1, most))
    batch = min(_log_int(rng, 1, 48), max(1, tokens // 2))
    while batch * max(qh, kh, vh) * dk * dv > 1 << 23:  # states no more than the packed prompts'
        batch = max(1, batch // 2)
    return dict(op=op, dtype=dtype, batch=batch, tokens=tokens, q_heads=qh, k_heads=kh, v_heads=vh, dk=dk, dv=dv,
                ragged=True, state=rng.random() < 0.5, fused=dk == dv and rng.random() < 0.5)


def draw(rng):
    op = rng.choice(("prefill", "prefill", "backward", "backward", "decode", "rotary", "rotary_backward"))
    if op in ("prefill", "backward"):
        return _draw_scan(rng, op)
    if op == "decode":
        dk, dv = rng.choice((16, 32, 48, 64, 80, 96, 128)), rng.choice((16, 32, 64, 96, 112, 128))
        qh, kh, vh = _draw_heads(rng, 64)
        batch = _log_int(rng, 1, max(1, min(1024, (1 << 26) // (max(qh, kh, vh) * dk * dv))))
        return dict(op=op, dtype=rng.choice(("bf16", "f32")), batch=batch, tokens=batch, q_heads=qh, k_heads=kh,
                    v_heads=vh, dk=dk, dv=dv, ragged=False, state=True, fused=dk == dv and rng.random() < 0.5,
                    pool=batch + rng.choice((0, 1, 7)), state_dtype=rng.choice(("f32", "f32", "bf16")))
    dim = rng.choice((16, 32, 48, 64, 80, 96, 128, 192, 256))
    rot = rng.choice((dim, dim, dim // 2))
    qh = rng.choice((1, 2, 3, 5, 8, 16, 28, 32, 64))
    kh = rng.choice([d for d in (1, 2, 4, 8, 32, 64) if d <= qh])
    most = min(1 << 15, (1 << 26) // ((qh + kh) * dim))
    return dict(op=op, dtype=rng.choice(("bf16", "bf16", "f32")), tokens=_log_int(rng, 1, most), q_heads=qh, k_heads=kh,
                dim=dim, rot=rot, axes=rng.choice((1, 1, 2, 3)), halves=rng.random() < 0.5,
                norm=rng.random() < 0.8, weight=rng.random() < 0.7, far=rng.random() < 0.3,
                fused=op == "rotary" and rng.random() < 0.5)


# ---- inputs ----------------------------------------------------------------

def _lengths(c):
    """Tokens of each sequence: the case's own, the same for every seed."""
    b, t = c["batch"], c["tokens"]
    if not c["ragged"] or b == 1:
        return [t // b + (i < t % b) for i in range(b)]
    r = np.random.RandomState((b * 65537 + t) % (1 << 31))
    fixed = [0, 1] if b >= 4 and t > 8 * b else []
    rest = r.multinomial(t - sum(fixed), r.dirichlet(np.full(b - len(fixed), 1.5)))
    return [int(n) for n in r.permutation(np.concatenate([fixed, rest]))]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    c, dt = dict(case), _DT[case["dtype"]]
    st = {"case": c}
    if c["op"].startswith("rotary"):
        T, qh, kh, d, ax, n = c["tokens"], c["q_heads"], c["k_heads"], c["dim"], c["axes"], c["rot"] // 2
        if c["fused"]:  # rows of one projection: queries, keys and a values part that stays unread
            rows = normal(T, qh + 2 * kh, d, dtype=dt)
            st["q"], st["k"] = rows[:, :qh], rows[:, qh:qh + kh]
        else:
            st["q"], st["k"] = normal(T, qh, d, dtype=dt), normal(T, kh, d, dtype=dt)
        freq = 10000.0 ** (-torch.arange(n, device="cuda", dtype=torch.float64) / n)
        part = torch.arange(n, device="cuda") * ax // n
        st["inv_freq"] = torch.stack([freq * (part == a) for a in range(ax)]).float()
        if c["far"]:
            pos = torch.randint(0, 1 << 20, (ax, T), generator=g, device="cuda")
        else:
            t = torch.arange(T, device="cuda") + torch.randint(0, 64, (1,), generator=g, device="cuda")
            pos = torch.stack([t // 1024, t // 32 % 32, t % 32][:ax]) if ax > 1 else t[None]
        st["positions"] = pos.to(torch.int64 if c["far"] else torch.int32).contiguous()
        st["q_weight"] = 1 + normal(d, std=0.25) if c["weight"] and c["norm"] else None
        st["k_weight"] = 1 + normal(d, std=0.25) if c["weight"] and c["norm"] else None
        if c["op"] == "rotary_backward":
            st["gq"], st["gk"] = normal(T, qh, d, dtype=dt), normal(T, kh, d, dtype=dt)
        return st
    T, B, qh, kh, vh, dk, dv = (c[k] for k in ("tokens", "batch", "q_heads", "k_heads", "v_heads", "dk", "dv"))
    H = max(qh, kh, vh)
    if c["fused"]:
        rows = normal(T, qh + kh + vh, dk, dtype=dt)
        st["q"], st["k"], st["v"] = rows[:, :qh], rows[:, qh:qh + kh], rows[:, qh + kh:]
    else:
        st["q"], st["k"], st["v"] = normal(T, qh, dk, dtype=dt), normal(T, kh, dk, dtype=dt), normal(T, vh, dv, dtype=dt)
    # from a memory of one or two tokens to one of hundreds, head by head
    jitter = 0.9 + 0.2 * torch.rand(H, generator=g, device="cuda")
    st["log_decay"] = -(2.0 ** (-8.0 * (torch.arange(H, device="cuda") + 1) / H)) * jitter
    if c["op"] == "decode":
        sd = _DT[c["state_dtype"]]
        st["state"] = normal(c["pool"], H, dk, dv, dtype=sd)
        st["slots"] = torch.randperm(c["pool"], generator=g, device="cuda")[:B].to(torch.int32)
        return st
    st["lengths"] = _lengths(c)
    st["cu_seqlens"] = torch.tensor(np.concatenate([[0], np.cumsum(st["lengths"])]), dtype=torch.int32, device="cuda")
    st["max_seqlen"] = max(st["lengths"])
    st["state"] = normal(B, H, dk, dv) if c["state"] else None
    if c["op"] == "backward":
        st["go"] = normal(T, H, dv, dtype=dt)
        st["gfinal"] = normal(B, H, dk, dv) if c["state"] else None
    return st


# ---- one pass --------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


def _own_prefill(st):
    from mamba_selective_ssm_ssd_amd import linear
    final = torch.empty_like(st["state"]) if st["state"] is not None else None
    o, final = linear.prefill(st["q"], st["k"], st["v"], st["log_decay"], state=st["state"], final=final,
                              cu_seqlens=st["cu_seqlens"], max_seqlen=st["max_seqlen"])
    return {"o": o, "state": final}


def _own_backward(st):
    from mamba_selective_ssm_ssd_amd import linear
    return linear.backward(st["q"], st["k"], st["v"], st["log_decay"], st["go"], state=st["state"],
                           gfinal=st["gfinal"], cu_seqlens=st["cu_seqlens"], max_seqlen=st["max_seqlen"])


def _own_decode(st):
    from mamba_selective_ssm_ssd_amd import linear
    o = linear.decode_step(st["q"], st["k"], st["v"], st["log_decay"], st["state"], slots=st["slots"])
    return {"o": o, "state": st["state"]}


def _own_rotary(st):
    from mamba_selective_ssm_ssd_amd import rotary
    c = st["case"]
    q, k = rotary.norm_rotate(st["q"], st["k"], st["positions"], st["inv_freq"], norm=c["norm"],
                              q_weight=st["q_weight"], k_weight=st["k_weight"], halves=c["halves"])
    return {"q": q, "k": k}


def _own_rotary_backward(st):
    from mamba_selective_ssm_ssd_amd import rotary
    c = st["case"]
    return rotary.norm_rotate_backward(st["q"], st["k"], st["positions"], st["inv_freq"], st["gq"], st["gk"],
                                       norm=c["norm"], q_weight=st["q_weight"], k_weight=st["k_weight"],
                                       halves=c["halves"])


def _per_head(x, heads):
    return x.float().repeat_interleave(heads // x.shape[1], dim=1)


def _chunk_rows(lengths, cu_seqlens, total, reverse):
    """Rows of every chunk [n, 64] (``total`` where there is none), its sequence, its place in it, its row count."""
    count = sum((n + _CHUNK - 1) // _CHUNK for n in lengths)
    dev = cu_seqlens.device
    start = cu_seqlens[:-1].long()
    length = cu_seqlens[1:].long() - start
    n = (length + _CHUNK - 1) // _CHUNK
    seq = torch.repeat_interleave(torch.arange(len(lengths), device=dev), n, output_size=count)
    place = torch.arange(count, device=dev) - (torch.cumsum(n, 0) - n)[seq]
    at = place[:, None] * _CHUNK + torch.arange(_CHUNK, device=dev)
    row = (length[seq][:, None] - 1 - at if reverse else at) + start[seq][:, None]
    rows = torch.where(at < length[seq][:, None], row, total)
    return rows, seq, place, (length[seq] - place * _CHUNK).clamp(max=_CHUNK)


def _scan(x, y, z, log_decay, st, init, reverse, a_in, a_init, a_state):
    """Chunked form of a decayed scan in 32 bits (decay factors from 64): with S the weighted sum of y z^T before a
    row, out = a_in (rows of its own chunk up to itself) + a_init (x S).  Reversed, S decays behind the row."""
    T, H, _ = x.shape
    rows, seq, place, count = _chunk_rows(st["lengths"], st["cu_seqlens"], T, reverse)
    e = 0 if reverse else 1
    ld = log_decay.double()

    def chunks(t):
        return torch.cat([t, t.new_zeros(1, *t.shape[1:])])[rows].permute(2, 0, 1, 3).contiguous()

    x, y, z = chunks(x), chunks(y), chunks(z)
    r = torch.arange(_CHUNK, device=x.device)
    mask = torch.exp(ld[:, None, None] * (r[:, None] - r).clamp(min=0)).float().tril()
    out = a_in * ((x @ y.transpose(2, 3).contiguous()) * mask[:, None]) @ z
    w = torch.exp(ld[:, None, None] * (count[:, None] - r - e).clamp(min=0)).float()
    U = a_state * (y * w[..., None]).transpose(2, 3).contiguous() @ z
    gap = place[:, None] - place - 1
    M = torch.exp(ld[:, None, None] * (_CHUNK * gap.clamp(min=0))).float() * ((seq[:, None] == seq) & (gap >= 0))
    S = (M @ U.flatten(2)).view_as(U)
    if init is not None:
        S += torch.exp(ld[:, None] * (_CHUNK * place)).float()[..., None, None] * init.float().transpose(0, 1)[:, seq]
    out += a_init * torch.exp(ld[:, None] * (r + e)).float()[:, None, :, None] * (x @ S)
    whole = out.new_zeros(T + 1, H, out.shape[-1])
    whole[rows.flatten()] = out.permute(1, 2, 0, 3).reshape(-1, H, out.shape[-1])
    end = torch.exp(ld[:, None] * count).float()[..., None, None] * S + U
    final = torch.zeros(len(st["lengths"]), *end.shape[:1], *end.shape[2:], device=x.device)
    if init is not None:
        final += init.float()
    last = place == torch.bincount(seq, minlength=len(st["lengths"]))[seq] - 1
    b = torch.where(last, seq, len(st["lengths"]))  # chunks before the last go to a row that is dropped
    final = torch.cat([final, final[:1]])
    final[b] = end.transpose(0, 1)
    return whole[:T], final[:-1]


def _plain_prefill(st):
    H = max(st["q"].shape[1], st["k"].shape[1], st["v"].shape[1])
    s = st["q"].shape[2] ** -0.5
    o, final = _scan(*(_per_head(st[n], H) for n in "qkv"), st["log_decay"], st, st["state"], False, s, s, 1.0)
    return {"o": o.to(st["q"].dtype), "state": final}


def _plain_backward(st):
    H = max(st["q"].shape[1], st["k"].shape[1], st["v"].shape[1])
    s, ld, dt = st["q"].shape[2] ** -0.5, st["log_decay"], st["q"].dtype
    q, k, v, go = (_per_head(st[n], H) for n in ("q", "k", "v", "go"))
    turned = [t.transpose(2, 3) if t is not None else None for t in (st["state"], st["gfinal"])]
    dq, _ = _scan(go, v, k, ld, st, turned[0], False, s, s, 1.0)
    dk, _ = _scan(v, go, q, ld, st, turned[1], True, s, 1.0, s)
    dv, first = _scan(k, q, go, ld, st, st["gfinal"], True, s, 1.0, s)
    grads = {n: d.view(d.shape[0], st[n].shape[1], -1, d.shape[2]).sum(2).to(dt) for n, d in zip("qkv", (dq, dk, dv))}
    if st["state"] is not None:
        grads["state"] = first
    return grads


def _plain_decode(st):
    H = st["state"].shape[1]
    q, k, v = (_per_head(st[n], H) for n in "qkv")
    at = st["slots"].long()
    S = torch.exp(st["log_decay"])[:, None, None] * st["state"][at].float() + k[..., None] * v[..., None, :]
    o = (q[..., None] * S).sum(2) * q.shape[2] ** -0.5
    st["state"][at] = S.to(st["state"].dtype)
    return {"o": o.to(st["q"].dtype), "state": st["state"]}


def _cos_sin(st):
    angle = (st["positions"].double()[..., None] * st["inv_freq"].double()[:, None]).sum(0)
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _turn(x, cos, sin, halves):
    n = cos.shape[-1]
    a, b = (x[..., :n], x[..., n:2 * n]) if halves else (x[..., 0:2 * n:2], x[..., 1:2 * n:2])
    pair = (a * cos - b * sin, a * sin + b * cos)
    return torch.cat([torch.cat(pair, -1) if halves else torch.stack(pair, -1).flatten(-2), x[..., 2 * n:]], -1)


def _plain_rotary(st):
    c, (cos, sin) = st["case"], _cos_sin(st)
    out = {}
    for n in "qk":
        x = st[n].float()
        if c["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
            x = x if st[n + "_weight"] is None else x * st[n + "_weight"]
        out[n] = _turn(x, cos, sin, c["halves"]).to(st[n].dtype)
    return out


def _plain_rotary_backward(st):
    c, (cos, sin) = st["case"], _cos_sin(st)
    out = {}
    for n in "qk":
        g = _turn(st["g" + n].float(), cos, -sin, c["halves"])
        if c["norm"]:
            x, w = st[n].float(), st[n + "_weight"]
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
            if w is not None:
                out[n + "_weight"] = (g * x * r).sum((0, 1))
                g = g * w
            g = r * g - r * r * r * x * (x * g).mean(-1, keepdim=True)
        out[n] = g.to(st[n].dtype)
    return out


_OWN = {"prefill": _own_prefill, "backward": _own_backward, "decode": _own_decode, "rotary": _own_rotary,
        "rotary_backward": _own_rotary_backward}
_PLAIN = {"prefill": _plain_prefill, "backward": _plain_backward, "decode": _plain_decode, "rotary": _plain_rotary,
          "rotary_backward": _plain_rotary_backward}


# ---- what a pass cannot do without -----------------------------------------

def work(case):
    c = case
    e = _SIZE[c["dtype"]]
    if c["op"].startswith("rotary"):
        rows = c["tokens"] * (c["q_heads"] + c["k_heads"]) * c["dim"]
        back = c["op"] == "rotary_backward"
        small = c["tokens"] * c["axes"] * (8 if c["far"] else 4) + c["axes"] * c["rot"] * 2
        # without a norm the gradient needs no x
        return {"bytes": rows * e * (3 if back and c["norm"] else 2) + small, "flops": rows * (14 if back else 7)}
    T, B, qh, kh, vh, dk, dv = (c[k] for k in ("tokens", "batch", "q_heads", "k_heads", "v_heads", "dk", "dv"))
    H = max(qh, kh, vh)
    rows_in, rows_out = T * ((qh + kh) * dk + vh * dv) * e, T * H * dv * e
    if c["op"] == "decode":
        return {"bytes": rows_in + rows_out + 2 * B * H * dk * dv * _SIZE[c["state_dtype"]] + 4 * B,
                "flops": 5 * B * H * dk * dv}
    states = 4 * B * H * dk * dv
    scan = T * H * (4 * dk * dv + _CHUNK * (dk + dv))  # two products with the state, half of the causal tile's two
    if c["op"] == "prefill":
        return {"bytes": rows_in + rows_out + states * (2 if c["state"] else 1), "flops": scan}
    return {"bytes": 2 * rows_in + rows_out + (3 * states if c["state"] else 0), "flops": 3 * scan}


# ---- the definition, token by token in 64 bits -----------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"prefill": _exact_scan, "backward": _exact_scan, "decode": _exact_decode, "rotary": _exact_rotary,
            "rotary_backward": _exact_rotary}[case["op"]](st)


def _exact_scan(st):
    """One token of every sequence at a time; a sequence that has ended keeps its state."""
    back = st["case"]["op"] == "backward"
    H, T = st["log_decay"].shape[0], st["q"].shape[0]
    group = {n: torch.arange(H, device="cuda") // (H // st[n].shape[1]) for n in "qkv"}
    g = torch.exp(st["log_decay"].double())[:, None, None]
    s = st["q"].shape[2] ** -0.5
    start, end = st["cu_seqlens"][:-1].long(), st["cu_seqlens"][1:].long()
    dk, dv, B = st["q"].shape[2], st["v"].shape[2], len(st["lengths"])
    zero = torch.zeros(B, H, dk, dv, dtype=torch.float64, device="cuda")
    S = st["state"].double() if st["state"] is not None else zero
    if not back:
        o = torch.zeros(T + 1, H, dv, dtype=torch.float64, device="cuda")
        for t in range(max(st["lengths"])):
            row = torch.where(start + t < end, start + t, T)
            q, k, v = (st[n][row.clamp(max=T - 1)].double()[:, group[n]] for n in "qkv")
            S = torch.where((row < T)[:, None, None, None], g * S + k[..., None] * v[:, :, None], S)
            o[row] = s * (q[:, :, None] @ S)[:, :, 0]
        return {"o": o[:T], "state": S}
    dq, dkk = (torch.zeros(T + 1, H, dk, dtype=torch.float64, device="cuda") for _ in range(2))
    dvv = torch.zeros(T + 1, H, dv, dtype=torch.float64, device="cuda")
    for t in range(max(st["lengths"])):
        row = torch.where(start + t < end, start + t, T)
        at = row.clamp(max=T - 1)
        k, v, go = st["k"][at].double()[:, group["k"]], st["v"][at].double()[:, group["v"]], st["go"][at].double()
        S = torch.where((row < T)[:, None, None, None], g * S + k[..., None] * v[:, :, None], S)
        dq[row] = s * (S @ go[..., None])[..., 0]
    G = st["gfinal"].double() if st["gfinal"] is not None else zero  # dL/dS behind the token, decayed after it
    for t in range(max(st["lengths"])):
        row = torch.where(end - 1 - t >= start, end - 1 - t, T)
        at = row.clamp(max=T - 1)
        q, k, v = (st[n][at].double()[:, group[n]] for n in "qkv")
        here = G + s * q[..., None] * st["go"][at].double()[:, :, None]
        dkk[row] = (here @ v[..., None])[..., 0]
        dvv[row] = (k[:, :, None] @ here)[:, :, 0]
        G = torch.where((row < T)[:, None, None, None], g * here, G)
    grads = {n: torch.zeros(T, *st[n].shape[1:], dtype=torch.float64, device="cuda").index_add_(1, group[n], d[:T])
             for n, d in zip("qkv", (dq, dkk, dvv))}
    if st["state"] is not None:
        grads["state"] = G
    return grads


def _exact_decode(st):
    H = st["log_decay"].shape[0]
    q, k, v = (st[n].double()[:, torch.arange(H, device="cuda") // (H // st[n].shape[1])] for n in "qkv")
    pool = st["state"].double()
    at = st["slots"].long()
    S = torch.exp(st["log_decay"].double()).view(1, H, 1, 1) * pool[at] + torch.einsum("bhk,bhv->bhkv", k, v)
    pool[at] = S
    return {"o": torch.einsum("bhk,bhkv->bhv", q, S) * q.shape[2] ** -0.5, "state": pool}


def _exact_rotary(st):
    """Pairs as complex numbers; the gradients by differentiating this definition."""
    c, n = st["case"], st["case"]["rot"] // 2
    p, f = st["positions"].double(), st["inv_freq"].double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.einsum("at,an->tn", p, f))[:, None]
    back = c["op"] == "rotary_backward"
    out = {}
    for name in "qk":
        x = st[name].double().requires_grad_(back)
        w = st[name + "_weight"]
        w = w.double().requires_grad_(back) if w is not None else None
        y = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() if c["norm"] else x
        y = y * w if w is not None else y
        head = y[..., :2 * n]
        z = head.unflatten(-1, (2, n)).transpose(-1, -2) if c["halves"] else head.unflatten(-1, (n, 2))
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
        y = torch.cat([z.transpose(-1, -2).flatten(-2) if c["halves"] else z.flatten(-2), y[..., 2 * n:]], -1)
        if not back:
            out[name] = y
            continue
        grads = torch.autograd.grad(y, [x] + ([w] if w is not None else []), st["g" + name].double())
        out[name] = grads[0]
        if w is not None:
            out[name + "_weight"] = grads[1]
    return out
