"""Linear attention with a decay for each head on the GPU against the fp64
oracle (oracle/linear.py): prompt pass, gradients, single-token step.

Tolerances.  Running the recurrence on absolute values gives, for every entry
of a result, the sum A of the sizes of its terms.  With bf16 I/O a term meets
at most one rounding of 2^-8 (of the entry of the chunk's starting state; the
weights q.k of its own chunk are held to 2^-17), and the result one more, so
|error| <= 2^-8 (A + |o|) up to second order.  fp32 results
(states, and everything with fp32 I/O) add about Dk + Dv + 64 + the number of
chunks terms in fp32, with decay factors of a few steps: at most 512 x 2^-24 A
for these sizes.
"""
import numpy as np
import pytest

from oracle import linear as ol

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U16, U32 = 2.0 ** -8, 512 * 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return t.double().cpu().numpy()


def _bound(A, out, dtype):
    return U32 * A + (1.01 * U16 * (A + np.abs(out)) if dtype == torch.bfloat16 else 0) + 1e-30


def _check(name, got, want, A, dtype):
    got = _np(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert np.isfinite(got).all(), f"{name}: not finite"
    over = np.abs(got - want) / _bound(A, want, dtype)
    worst = float(over.max()) if over.size else 0.0
    n = np.linalg.norm(want)
    rel = float(np.linalg.norm(got - want) / n) if n else 0.0
    print(f"{name}: {worst:.3f} of the bound, relative {rel:.2e}", flush=True)
    assert worst <= 1.0, name


class Case:
    """Inputs on the device and, rounded to their type, in fp64."""

    def __init__(self, lengths, heads, dk, dv, io, seed=0, state=False, sd=torch.float32, decay=(0.002, 0.7), fused=False):
        g = torch.Generator().manual_seed(seed)
        T, H = sum(lengths), max(heads)
        dt = DT[io]
        if fused:
            assert dk == dv
            rows = torch.randn(T, sum(heads), dk, generator=g).to(dt).cuda()
            self.q, self.k, self.v = rows.split(heads, dim=1)
        else:
            self.q, self.k, self.v = (torch.randn(T, h, d, generator=g).to(dt).cuda()
                                      for h, d in zip(heads, (dk, dk, dv)))
        self.go = torch.randn(T, H, dv, generator=g).to(dt).cuda()
        self.ld = -torch.exp(torch.empty(H).uniform_(np.log(decay[0]), np.log(decay[1]), generator=g)).cuda()
        self.cu = [0, *np.cumsum(lengths).tolist()]
        self.cu_dev = torch.tensor(self.cu, dtype=torch.int32, device="cuda")
        shape = (len(lengths), H, dk, dv)
        self.state = torch.randn(shape, generator=g).to(sd).cuda() if state else None
        self.gfinal = torch.randn(shape, generator=g).cuda() if state else None
        self.dt, self.lengths = dt, lengths

    def args(self):
        return self.q, self.k, self.v, self.ld

    def host(self, absolute=False):
        f = (lambda t: np.abs(_np(t))) if absolute else _np
        return [f(t) for t in (self.q, self.k, self.v)] + [_np(self.ld)]


def _run_prefill(c, **kw):
    from mamba_selective_ssm_ssd_amd import linear
    final = torch.empty_like(c.state) if c.state is not None else None
    o, final = linear.prefill(*c.args(), state=c.state, final=final, cu_seqlens=c.cu_dev, **kw)
    torch.cuda.synchronize()
    return o, final


def _oracle_prefill(c):
    s, sa = (None, None) if c.state is None else (_np(c.state), np.abs(_np(c.state)))
    return ol.prefill(*c.host(), c.cu, s), ol.prefill(*c.host(True), c.cu, sa)


def _check_prefill(c, **kw):
    o, final = _run_prefill(c, **kw)
    (wo, wf), (ao, af) = _oracle_prefill(c)
    _check("o", o, wo, ao, c.dt)
    _check("final", final, wf, af, final.dtype)


HEADS = [(3, 3, 3), (4, 2, 1), (1, 1, 4), (2, 6, 3)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(8, 8), (16, 40), (32, 32), (64, 64), (64, 128), (128, 64), (96, 80), (128, 128), (32, 128), (128, 24)])
def test_prefill_sizes(io, dk, dv):
    _check_prefill(Case([70, 1, 0, 33], (2, 2, 2), dk, dv, io, seed=dk + dv, state=True))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200])
def test_prefill_lengths(io, n):
    _check_prefill(Case([n], (2, 1, 2), 64, 32, io, seed=n, state=n % 2 == 1), max_seqlen=n)


@pytest.mark.parametrize("dk,dv", [(16, 24), (64, 64), (128, 128), (64, 128), (128, 32)])
@pytest.mark.parametrize("heads", [(2, 2, 2), (320, 320, 320)])
def test_few_tokens_round_once(dk, dv, heads):
    """Within a chunk the weights are held to 2^-17: without a state to start
    from, a bf16 result and its gradients meet one rounding, the result's own."""
    from mamba_selective_ssm_ssd_amd import linear
    c = Case([1, 2, 5], heads, dk, dv, "bf16", seed=dk + heads[0])
    o, _ = linear.prefill(*c.args(), cu_seqlens=c.cu_dev, max_seqlen=5)
    g = linear.backward(*c.args(), c.go, cu_seqlens=c.cu_dev, max_seqlen=5)
    want, size = [ol.prefill(*c.host(a), c.cu, None)[0] for a in (False, True)]
    wg = ol.backward(*c.host(), _np(c.go), c.cu, None, None)
    sg = ol.backward(*c.host(True), np.abs(_np(c.go)), c.cu, None, None)
    for name, got, w, a in (("o", o, want, size), *(("d" + n, g[n], wg[i], sg[i]) for i, n in enumerate("qkv"))):
        over = np.abs(_np(got) - w) / (1.01 * U16 * np.abs(w) + (2.0 ** -16 + U32) * a + 1e-30)
        print(f"{name}: {float(over.max()):.3f} of the bound", flush=True)
        assert float(over.max()) <= 1.0, name


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("heads", HEADS)
def test_prefill_head_groups(io, heads):
    _check_prefill(Case([65, 40], heads, 64, 64, io, seed=7, state=True, fused=True))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[1500], [700, 0, 1, 900, 257], [256, 512, 1024], [5, 1300, 63]])
@pytest.mark.parametrize("state", [False, True])
def test_prefill_cut_sequences(io, lengths, state):
    from mamba_selective_ssm_ssd_amd import capi, linear
    c = Case(lengths, (2, 2, 2), 64, 64, io, seed=sum(lengths), state=state)
    rc, seg, _ = capi.m3_linear_plan(linear.make_shape(len(lengths), sum(lengths), 2, 2, 2, 64, 64, c.dt))
    assert rc == 0 and 0 < seg < max(lengths)
    _check_prefill(c)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(16, 24), (64, 64), (64, 128), (128, 64), (128, 128), (32, 104)])
@pytest.mark.parametrize("lengths,heads", [([70, 1, 0, 33, 130], (6, 2, 6)), ([300, 0, 0, 270], (6, 6, 3))])
def test_many_heads(io, dk, dv, lengths, heads):
    """Workgroups enough for the widest column tiles, of whole sequences and cut
    ones: ten times the same heads, which have to agree bit for bit."""
    import copy
    from mamba_selective_ssm_ssd_amd import capi, linear
    c = Case(lengths, heads, dk, dv, io, seed=dk + dv, state=True)
    many, n = copy.copy(c), 10
    for name in ("q", "k", "v", "go", "state", "gfinal"):
        setattr(many, name, getattr(c, name).repeat(1, n, *[1] * (getattr(c, name).dim() - 2)))
    many.ld = c.ld.repeat(n)
    rc, a, b = capi.m3_linear_plan(linear.make_shape(len(lengths), sum(lengths), *(n * h for h in heads), dk, dv, c.dt, max_seqlen=max(lengths)))
    assert rc == 0 and (a > 0) == (b > 0) == (max(lengths) > 256)
    o, final = _run_prefill(many, max_seqlen=max(lengths))
    g = _run_backward(many, max_seqlen=max(lengths))
    for t, h in ((o, 6), (final, 6), *((g[x], heads["qkv".index(x)]) for x in "qkv"), (g["state"], 6)):
        assert all(torch.equal(t[:, i * h:(i + 1) * h], t[:, :h]) for i in range(1, n))
    (wo, wf), (ao, af) = _oracle_prefill(c)
    _check("o", o[:, :6], wo, ao, c.dt)
    _check("final", final[:, :6], wf, af, torch.float32)
    _compare_backward(c, {x: t[:, :heads["qkv".index(x)] if x != "state" else 6] for x, t in g.items()})


@pytest.mark.parametrize("state", [False, True])
def test_prefill_hint_changes_nothing_but_rounding(state):
    """max_seqlen is only a hint: too small, too large or absent."""
    c = Case([600, 900], (2, 2, 2), 64, 64, "bf16", seed=3, state=state)
    for hint in (None, 1, 600, 900, 100000):
        _check_prefill(c, max_seqlen=hint)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prefill_decays_at_the_ends(io):
    """No decay, a slow one over many chunks, a fast one, and one that forgets everything."""
    c = Case([1100], (5, 5, 5), 32, 32, io, seed=4, state=True)
    c.ld[:] = torch.tensor([0.0, -1e-6, -1e-3, -20.0, -float("inf")])
    _check_prefill(c)
    _check_backward(c)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prefill_dense_and_bf16_states(io):
    from mamba_selective_ssm_ssd_amd import linear
    c = Case([90, 90, 90], (4, 2, 4), 64, 64, io, seed=5, state=True, sd=torch.bfloat16)
    dense = [t.view(3, 90, *t.shape[1:]) for t in (c.q, c.k, c.v)]
    final = torch.empty_like(c.state)
    o, _ = linear.prefill(*dense, c.ld, state=c.state, final=final)
    assert o.shape == (3, 90, 4, 64) and final.dtype == torch.bfloat16
    (wo, wf), (ao, af) = _oracle_prefill(c)
    _check("o", o.flatten(0, 1), wo, ao, c.dt)
    # the bf16 state is one rounding of the fp32 one
    assert (np.abs(_np(final) - wf) <= 1.01 * U16 * np.abs(wf) + U32 * af).all()


def test_prefill_in_place_state_and_slots():
    from mamba_selective_ssm_ssd_amd import linear
    for lengths in ([40, 0, 70, 1], [700, 0, 900, 1]):
        c = Case(lengths, (2, 2, 2), 64, 64, "bf16", seed=6, state=True)
        pool = torch.randn(9, 2, 64, 64, device="cuda")
        slots = torch.tensor([7, 0, 3, 5], dtype=torch.int32, device="cuda")
        pool[slots.long()] = c.state
        before = pool.clone()
        o, out = linear.prefill(*c.args(), state=pool, cu_seqlens=c.cu_dev, slots=slots)
        assert out is pool
        (wo, wf), (ao, af) = _oracle_prefill(c)
        _check("o", o, wo, ao, c.dt)
        _check("final", pool[slots.long()], wf, af, torch.float32)
        rest = [1, 2, 4, 6, 8]
        assert torch.equal(pool[rest], before[rest])


def test_prefill_padding_slots_tail_rows_and_repeated_slots():
    from mamba_selective_ssm_ssd_amd import linear
    for lengths in ([40, 30, 70, 20], [400, 300, 700, 600]):
        c = Case(lengths, (2, 2, 2), 64, 64, "bf16", seed=8, state=True)
        T = sum(lengths)
        q, k, v = (torch.cat([t, torch.full_like(t[:5], float("nan"))]) for t in (c.q, c.k, c.v))
        pool = torch.randn(6, 2, 64, 64, device="cuda")
        slots = torch.tensor([4, -1, 4, 99], dtype=torch.int32, device="cuda")
        pool[4] = c.state[0]
        before = pool.clone()
        o = torch.full((T + 5, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16)
        linear.prefill(q, k, v, c.ld, state=pool, cu_seqlens=c.cu_dev, slots=slots, o=o)
        (wo, wf), (ao, af) = _oracle_prefill(c)
        a, b, d = c.cu[1], c.cu[2], c.cu[3]
        _check("o", o[:a], wo[:a], ao[:a], c.dt)
        assert (o[a:b] == 7).all() and torch.isnan(o[b:d].float()).all() and (o[d:] == 7).all()
        _check("state", pool[4], wf[0], af[0], torch.float32)
        rest = [0, 1, 2, 3, 5]
        assert torch.equal(pool[rest], before[rest])


def _run_backward(c, **kw):
    from mamba_selective_ssm_ssd_amd import linear
    g = linear.backward(*c.args(), c.go, state=c.state, gfinal=c.gfinal, cu_seqlens=c.cu_dev, **kw)
    torch.cuda.synchronize()
    return g


def _check_backward(c, **kw):
    _compare_backward(c, _run_backward(c, **kw))


def _compare_backward(c, g):
    pick = (lambda f: [None if t is None else f(_np(t)) for t in (c.state, c.gfinal)])
    want = ol.backward(*c.host(), _np(c.go), c.cu, *pick(lambda x: x))
    size = ol.backward(*c.host(True), np.abs(_np(c.go)), c.cu, *pick(np.abs))
    for i, n in enumerate("qkv"):
        assert g[n].dtype == c.dt
        _check("d" + n, g[n], want[i], size[i], c.dt)
    if c.state is not None:
        _check("dstate", g["state"], want[3], size[3], torch.float32)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(8, 16), (32, 32), (64, 64), (64, 128), (128, 64), (96, 80), (128, 128), (24, 128)])
def test_backward_sizes(io, dk, dv):
    _check_backward(Case([70, 1, 0, 33], (2, 2, 2), dk, dv, io, seed=dk + dv, state=True))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("heads", HEADS)
def test_backward_head_groups(io, heads):
    _check_backward(Case([65, 40], heads, 64, 64, io, seed=9, state=heads[0] != 3, fused=True))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[1500], [700, 0, 1, 900, 257]])
@pytest.mark.parametrize("state", [False, True])
def test_backward_cut_sequences(io, lengths, state):
    from mamba_selective_ssm_ssd_amd import capi, linear
    c = Case(lengths, (2, 2, 2), 64, 64, io, seed=10, state=state)
    rc, _, seg = capi.m3_linear_plan(linear.make_shape(len(lengths), sum(lengths), 2, 2, 2, 64, 64, c.dt))
    assert rc == 0 and 0 < seg < max(lengths)
    _check_backward(c)


@pytest.mark.parametrize("heads", [(2, 2, 2), (2, 1, 1)])
def test_backward_rows_outside_every_sequence_are_zero(heads):
    from mamba_selective_ssm_ssd_amd import linear
    c = Case([30, 40], heads, 64, 64, "bf16", seed=11)
    pad = lambda t: torch.cat([t[:3], t, t[:9]])  # noqa: E731
    cu = c.cu_dev + 3
    g = linear.backward(pad(c.q), pad(c.k), pad(c.v), c.ld, pad(c.go), cu_seqlens=cu)
    ref = linear.backward(*c.args(), c.go, cu_seqlens=c.cu_dev)
    for n in "qkv":
        assert torch.equal(g[n][3:73], ref[n]) and not g[n][:3].any() and not g[n][73:].any()


def test_backward_matches_differences_of_the_kernel_itself():
    """A directional difference of the fp32 prompt pass."""
    from mamba_selective_ssm_ssd_amd import linear
    c = Case([50, 300], (2, 1, 2), 32, 48, "f32", seed=12, state=True, decay=(0.05, 0.7))

    def loss(q, k, v, s):
        o, f = linear.prefill(q, k, v, c.ld, state=s, final=torch.empty_like(s), cu_seqlens=c.cu_dev)
        return float((o.double() * c.go.double()).sum() + (f.double() * c.gfinal.double()).sum())

    g = _run_backward(c)
    x = [c.q, c.k, c.v, c.state]
    for i, n in enumerate(("q", "k", "v", "state")):
        d = torch.randn(x[i].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(i))
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + 0.25 * d, x[i] - 0.25 * d
        # o is linear in each operand: the difference is exact but for fp32 rounding
        diff, want = (loss(*up) - loss(*down)) / 0.5, float((g[n].double() * d.double()).sum())
        assert abs(diff - want) <= 1e-4 * float((g[n].double() * d.double()).abs().sum()), (n, diff, want)


def _oracle_step(c, pool, slots):
    q, k, v, ld = c.host()
    cu = list(range(len(slots) + 1))
    ok = [ol.prefill(*x, cu, s) for x, s in (((q, k, v, ld), pool[slots]), ((*(abs(t) for t in (q, k, v)), ld), abs(pool[slots])))]
    return ok


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("sd", ["f32", "bf16"])
@pytest.mark.parametrize("B,heads,dk,dv", [(1, (1, 1, 1), 8, 8), (3, (4, 2, 1), 64, 64), (5, (2, 2, 2), 128, 128), (2, (3, 3, 3), 96, 80),
                                           (70, (2, 4, 16), 32, 72), (130, (8, 8, 8), 64, 128), (300, (4, 1, 4), 16, 8)])
def test_decode_step(io, sd, B, heads, dk, dv):
    from mamba_selective_ssm_ssd_amd import linear
    c = Case([1] * B, heads, dk, dv, io, seed=B, fused=dk == dv)
    H = max(heads)
    pool = torch.randn(B + 3, H, dk, dv, generator=torch.Generator().manual_seed(B)).to(DT[sd]).cuda()
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(1))[:B]
    before = pool.clone()
    o = linear.decode_step(*c.args(), pool, slots=slots.int().cuda())
    (wo, wf), (ao, af) = _oracle_step(c, _np(before), slots.numpy())
    # fp32 arithmetic throughout: only the result is rounded
    assert (np.abs(_np(o) - wo) <= U32 * ao + (1.01 * U16 * np.abs(wo) if io == "bf16" else 0)).all()
    assert (np.abs(_np(pool[slots.cuda()]) - wf) <= U32 * af + (1.01 * U16 * np.abs(wf) if sd == "bf16" else 0)).all()
    rest = [i for i in range(B + 3) if i not in set(slots.tolist())]
    assert torch.equal(pool[rest], before[rest])
    # without slots: the first B states
    pool = before.clone()
    o2 = linear.decode_step(*c.args(), pool[:B])
    (wo, wf), (ao, af) = _oracle_step(c, _np(before), np.arange(B))
    assert (np.abs(_np(o2) - wo) <= U32 * ao + (1.01 * U16 * np.abs(wo) if io == "bf16" else 0)).all()
    assert torch.equal(pool[B:], before[B:])


def test_decode_step_padding_and_repeated_slots():
    from mamba_selective_ssm_ssd_amd import linear
    c = Case([1] * 6, (2, 2, 2), 64, 64, "bf16", seed=20)
    pool = torch.randn(4, 2, 64, 64, device="cuda")
    before = pool.clone()
    slots = torch.tensor([2, -1, 2, 0, 4, 0], dtype=torch.int32, device="cuda")
    o = torch.full((6, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    linear.decode_step(*c.args(), pool, slots=slots, o=o)
    ref = before.clone()
    o_ref = linear.decode_step(*(t[[0, 3]] for t in c.args()[:3]), c.ld, ref, slots=slots[[0, 3]].contiguous())
    assert torch.equal(pool, ref) and torch.equal(o[[0, 3]], o_ref)
    assert (o[[1, 4]] == 7).all() and torch.isnan(o[[2, 5]].float()).all()


def test_slow_decay_over_many_steps():
    """4000 steps of a decay so slow that rounding it to 24 bits would show."""
    from mamba_selective_ssm_ssd_amd import linear
    ld = torch.tensor([-1e-5], device="cuda")
    pool = torch.ones(1, 1, 32, 32, device="cuda")
    z = torch.zeros(1, 1, 32, device="cuda")
    for _ in range(4000):
        linear.decode_step(z, z, z, ld, pool)
    want = float(np.exp(float(ld[0]) * 4000.0))
    # one fma of half a step per token: 4000 x 2^-25 as a walk, 4 sigma
    assert abs(float(pool.double().mean()) - want) <= 4 * np.sqrt(4000.0) * 2.0 ** -25
    ones = torch.ones(1, 1, 32, 32, device="cuda")
    zz = torch.zeros(60000, 1, 32, device="cuda")
    _, f = linear.prefill(zz, zz, zz, ld, state=ones, final=torch.empty_like(ones))
    want = float(np.exp(float(ld[0]) * 60000.0))
    assert abs(float(f.double().mean()) - want) <= 4 * np.sqrt(2000.0) * 2.0 ** -24


def test_prompt_then_steps_is_the_longer_prompt():
    """The operators together, as a layer uses them: rows normed and turned,
    the prompt, then token by token."""
    from mamba_selective_ssm_ssd_amd import linear, rotary
    T, n, H, D = 150, 130, 4, 64
    g = torch.Generator().manual_seed(30)
    qkv = torch.randn(T, 3 * H, D, generator=g).to(torch.bfloat16).cuda()
    q, k, v = qkv.split(H, dim=1)
    ld = -torch.tensor([0.5, 0.1, 0.02, 0.004], device="cuda")
    freq = 10000.0 ** (-torch.arange(32, device="cuda") / 32.0)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    qr, kr = rotary.norm_rotate(q, k, pos, freq)
    whole, end = linear.prefill(qr, kr, v, ld)
    qp, kp = rotary.norm_rotate(q[:n], k[:n], pos[:n], freq)
    o, state = linear.prefill(qp, kp, v[:n], ld)
    rows = [o]
    for t in range(n, T):
        qs, ks = rotary.norm_rotate(q[t:t + 1], k[t:t + 1], pos[t:t + 1], freq)
        rows.append(linear.decode_step(qs, ks, v[t:t + 1], ld, state))
    wo, wf = ol.prefill(_np(qr), _np(kr), _np(v), _np(ld), [0, T])
    ao, af = ol.prefill(*(np.abs(_np(t)) for t in (qr, kr, v)), _np(ld), [0, T])
    _check("prompt", whole, wo, ao, torch.bfloat16)
    _check("pieces", torch.cat(rows), wo, ao, torch.bfloat16)
    _check("end", end, wf, af, torch.float32)
    _check("state", state, wf, af, torch.float32)


def test_non_finite_tokens_stay_in_sequence_head_and_behind_their_chunk():
    c = Case([200, 700], (3, 3, 3), 64, 64, "bf16", seed=13)
    o0, f0 = _run_prefill(c)
    for bad in (float("nan"), float("inf")):
        for t in (70, 200 + 333):
            v = c.v.clone()
            c.v = v.clone()
            c.v[t, 1, 5] = bad
            o1, f1 = _run_prefill(c)
            c.v = v
            b = int(t >= 200)
            lo = c.cu[b] + (t - c.cu[b]) // 64 * 64
            same = torch.ones_like(o0, dtype=torch.bool)
            same[lo:c.cu[b + 1], 1, 5] = False
            assert torch.equal(o0[same], o1[same])
            assert not torch.isfinite(o1[t:c.cu[b + 1], 1, 5].float()).any()
            same = torch.ones_like(f0, dtype=torch.bool)
            same[b, 1, :, 5] = False
            assert torch.equal(f0[same], f1[same])


def test_results_do_not_depend_on_the_run_or_the_neighbours():
    """Bit for bit: twice the same call, on another stream, with garbage in the workspace."""
    from mamba_selective_ssm_ssd_amd import linear
    c = Case([700, 90, 300], (4, 2, 2), 64, 64, "bf16", seed=14, state=True)
    o0, f0 = _run_prefill(c)
    g0 = _run_backward(c)
    ws = torch.full((linear.workspace_bytes(c.q, c.k, c.v, c.cu_dev),), 255, dtype=torch.uint8, device="cuda")
    wb = torch.full((linear.workspace_bytes(c.q, c.k, c.v, c.cu_dev, backward=True),), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o1, f1 = _run_prefill(c, workspace=ws)
        g1 = _run_backward(c, workspace=wb)
    assert torch.equal(o0, o1) and torch.equal(f0, f1) and all(torch.equal(g0[n], g1[n]) for n in g0)


def test_two_streams_at_once():
    """Calls of two streams, each with a workspace of its own, beside each other."""
    from mamba_selective_ssm_ssd_amd import linear
    cases = [Case([900, 40, 700], (8, 4, 4), 64, 64, "bf16", seed=40, state=True), Case([1300], (6, 6, 6), 128, 128, "bf16", seed=41, state=True)]
    want = [(_run_prefill(c), _run_backward(c)) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                final = torch.empty_like(c.state)
                o, _ = linear.prefill(*c.args(), state=c.state, final=final, cu_seqlens=c.cu_dev)
                g = linear.backward(*c.args(), c.go, state=c.state, gfinal=c.gfinal, cu_seqlens=c.cu_dev)
                got[i].append((o, final, g))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for o, final, g in runs:
            assert torch.equal(o, w[0][0]) and torch.equal(final, w[0][1]) and all(torch.equal(g[n], w[1][n]) for n in g)


def test_two_graphs_that_share_a_workspace():
    from mamba_selective_ssm_ssd_amd import linear
    a = Case([900, 40], (4, 2, 2), 64, 64, "bf16", seed=42, state=True)
    b = Case([500, 600], (2, 2, 2), 128, 64, "bf16", seed=43, state=True)
    ws = torch.empty(max(linear.workspace_bytes(c.q, c.k, c.v, c.cu_dev, backward=r) for c in (a, b) for r in (False, True)),
                     dtype=torch.uint8, device="cuda")

    def work(c):
        o, f = linear.prefill(*c.args(), state=c.state, final=torch.empty_like(c.state), cu_seqlens=c.cu_dev, workspace=ws)
        return [o, f, *linear.backward(*c.args(), c.go, state=c.state, gfinal=c.gfinal, cu_seqlens=c.cu_dev, workspace=ws).values()]

    want = [[t.clone() for t in work(c)] for c in (a, b)]
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    torch.cuda.synchronize()
    for g, c in zip(graphs, (a, b)):
        with torch.cuda.graph(g):
            outs.append(work(c))
    for _ in range(3):
        for out in outs:
            for t in out:
                t.fill_(float("nan"))
        ws.fill_(255)
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for out, w in zip(outs, want) for x, y in zip(out, w))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_strides_broadcasts_and_a_start_behind_zero(io):
    """Rows as [head][token][channel], heads broadcast by a stride of zero, sequences that start behind row 0."""
    from mamba_selective_ssm_ssd_amd import linear
    c = Case([300, 20], (4, 2, 4), 64, 32, io, seed=44, state=True)
    o0, f0 = _run_prefill(c)
    g0 = _run_backward(c)
    turn = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    o1 = torch.empty(4, 320, 32, device="cuda", dtype=c.dt).transpose(0, 1)
    f1 = torch.empty_like(f0)
    linear.prefill(turn(c.q), turn(c.k), turn(c.v), c.ld, state=c.state, final=f1, cu_seqlens=c.cu_dev, o=o1)
    g1 = linear.backward(turn(c.q), turn(c.k), turn(c.v), c.ld, turn(c.go), state=c.state, gfinal=c.gfinal, cu_seqlens=c.cu_dev)
    assert torch.equal(o0, o1) and torch.equal(f0, f1) and all(torch.equal(g0[n], g1[n]) for n in g0)
    one = c.k[:, :1]
    oa, _ = linear.prefill(c.q, one.expand(320, 4, 64), c.v, c.ld, cu_seqlens=c.cu_dev)
    ob, _ = linear.prefill(c.q, one.repeat(1, 4, 1), c.v, c.ld, cu_seqlens=c.cu_dev)
    assert torch.equal(oa, ob)
    pad = lambda t: torch.cat([torch.full_like(t[:7], float("nan")), t, torch.full_like(t[:9], float("nan"))])  # noqa: E731
    o2 = torch.full((336, 4, 32), 5.0, device="cuda", dtype=c.dt)
    f2 = torch.empty_like(f0)
    linear.prefill(pad(c.q), pad(c.k), pad(c.v), c.ld, state=c.state, final=f2, cu_seqlens=c.cu_dev + 7, o=o2)
    # where a segment starts depends on the first row's number: up to rounding the same
    (wo, wf), (ao, af) = _oracle_prefill(c)
    _check("o", o2[7:327], wo, ao, c.dt)
    _check("final", f2, wf, af, torch.float32)
    assert (o2[:7] == 5).all() and (o2[327:] == 5).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rows_as_far_apart_as_strides_go(io):
    """The widest stride of tokens: a chunk spans 2 GiB, all rows many."""
    from mamba_selective_ssm_ssd_amd import linear, rotary
    T, H, D, wide = 270, 2, 64, (1 << 24) - 8
    c = Case([T], (H, H, H), D, D, io, seed=48, state=True)
    flat = torch.empty((T - 1) * wide + 6 * H * D, device="cuda", dtype=c.dt)

    def far(i, t=None):
        v = flat[i * H * D:].as_strided((T, H, D), (wide, D, 1))
        if t is not None:
            v.copy_(t)
        return v

    q, k, v, go, o = far(0, c.q), far(1, c.k), far(2, c.v), far(3, c.go), far(4)
    want, final = _run_prefill(c)
    got, f = linear.prefill(q, k, v, c.ld, state=c.state, final=torch.empty_like(final), o=o)
    assert torch.equal(got, want) and torch.equal(f, final)
    ref = _run_backward(c)
    g = linear.backward(q, k, v, c.ld, go, state=c.state, gfinal=c.gfinal)
    assert all(torch.equal(g[n], ref[n]) for n in ref)
    pos, freq = torch.arange(T, device="cuda", dtype=torch.int32), torch.linspace(1, 0.01, 32, device="cuda")
    a = rotary.norm_rotate(c.q, c.k, pos, freq)
    b = rotary.norm_rotate(q, k, pos, freq, q_out=q, k_out=k)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(v, c.v) and torch.equal(go, c.go)
    with pytest.raises(Exception):
        linear.prefill(flat.as_strided((2, H, D), (1 << 24, D, 1)), c.k[:2], c.v[:2], c.ld)


def test_no_tokens_at_all():
    from mamba_selective_ssm_ssd_amd import linear
    c = Case([0, 0, 0], (4, 2, 1), 64, 32, "bf16", seed=45, state=True)
    o, f = _run_prefill(c)
    assert o.shape == (0, 4, 32) and torch.equal(f, c.state)
    g = _run_backward(c)
    assert g["k"].shape == (0, 2, 64) and torch.equal(g["state"], c.gfinal)
    with pytest.raises(Exception):
        linear.decode_step(*c.args(), c.state[:0])


def test_states_larger_than_32_bits_count():
    """A pool of more than 2^31 entries: the last states of it, prompt and step."""
    from mamba_selective_ssm_ssd_amd import linear
    n = (1 << 31) // (4 * 128 * 128) + 3
    pool = torch.empty(n, 4, 128, 128, device="cuda")
    c = Case([70, 40], (4, 2, 2), 128, 128, "bf16", seed=46, state=True)
    slots = torch.tensor([n - 1, n - 2], dtype=torch.int32, device="cuda")
    pool[[n - 1, n - 2]] = c.state
    pool[[0, n - 3]] = 3.0
    o, _ = linear.prefill(*c.args(), state=pool, cu_seqlens=c.cu_dev, slots=slots)
    o1, f1 = _run_prefill(c)
    assert torch.equal(o, o1) and torch.equal(pool[[n - 1, n - 2]], f1)
    d = Case([1, 1], (4, 2, 2), 128, 128, "bf16", seed=47)
    s = linear.decode_step(*d.args(), pool, slots=slots)
    assert torch.equal(s, linear.decode_step(*d.args(), f1)) and torch.equal(pool[[n - 1, n - 2]], f1)
    assert (pool[[0, n - 3]] == 3).all()


def test_graph_capture_and_replay():
    from mamba_selective_ssm_ssd_amd import linear, rotary
    c = Case([600, 0, 300], (4, 2, 2), 64, 64, "bf16", seed=15, state=True)
    d = Case([1, 1, 1], (4, 2, 2), 64, 64, "bf16", seed=16)
    freq = 10000.0 ** (-torch.arange(32, device="cuda") / 32.0)
    pos = torch.arange(900, device="cuda", dtype=torch.int32)
    w = torch.linspace(0.5, 1.5, 64, device="cuda")
    final, pool = torch.empty_like(c.state), c.state.clone()

    def work():
        q, k = rotary.norm_rotate(c.q, c.k, pos, freq, q_weight=w, k_weight=w)
        o, _ = linear.prefill(q, k, c.v, c.ld, state=c.state, final=final, cu_seqlens=c.cu_dev)
        g = linear.backward(q, k, c.v, c.ld, c.go, state=c.state, gfinal=c.gfinal, cu_seqlens=c.cu_dev)
        r = rotary.norm_rotate_backward(c.q, c.k, pos, freq, g["q"], g["k"], q_weight=w, k_weight=w)
        s = linear.decode_step(*d.args(), pool)
        return [o, final, s, *g.values(), *r.values()]

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for i in range(3):
        c.q.normal_(generator=torch.Generator("cuda").manual_seed(i))
        pool.copy_(c.state)
        want = [t.clone() for t in work()]
        pool.copy_(c.state)
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_device_refusals():
    from mamba_selective_ssm_ssd_amd import capi, linear
    c = Case([10], (2, 2, 2), 64, 64, "bf16", seed=17)
    with pytest.raises(capi.M3Error):                                   # rows that are not 16-byte aligned
        linear.prefill(torch.randn(10, 2, 65, device="cuda").bfloat16()[..., 1:], c.k, c.v, c.ld)
    with pytest.raises(ValueError):                                     # channels with a stride
        linear.prefill(torch.randn(10, 2, 128, device="cuda").bfloat16()[..., ::2], c.k, c.v, c.ld)
    with pytest.raises(capi.M3Error):                                   # a head count that does not divide
        linear.prefill(c.q, c.k, torch.randn(10, 3, 64, device="cuda").bfloat16(),
                       torch.zeros(3, device="cuda"))
    with pytest.raises(capi.M3Error):                                   # a size outside the set
        linear.prefill(torch.randn(10, 2, 136, device="cuda").bfloat16(), torch.randn(10, 2, 136, device="cuda").bfloat16(), c.v, c.ld)
    with pytest.raises(capi.M3Error):
        linear.prefill(*c.args(), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    for kw in (dict(o=torch.empty(9, 2, 64, device="cuda", dtype=torch.bfloat16)), dict(state=torch.zeros(2, 2, 64, 64, device="cuda")),
               dict(cu_seqlens=torch.tensor([0, 10], device="cuda")), dict(cu_seqlens=torch.tensor([0, 10], dtype=torch.int32)),
               dict(slots=torch.zeros(1, dtype=torch.int32, device="cuda")), dict(state=torch.zeros(1, 2, 64, 64, device="cuda", dtype=torch.float16))):
        with pytest.raises(ValueError):
            linear.prefill(*c.args(), **kw)
    with pytest.raises(ValueError):
        linear.prefill(c.q.cpu(), c.k, c.v, c.ld)
    with pytest.raises(ValueError):
        linear.prefill(c.q, c.k.float(), c.v, c.ld)
    with pytest.raises(ValueError):
        linear.backward(*c.args(), c.go[:5])
    with pytest.raises(capi.M3Error):                                   # an output that is an input
        linear.prefill(*c.args(), o=c.v)
    with pytest.raises(capi.M3Error):                                   # outputs that overlap themselves
        linear.prefill(*c.args(), o=torch.empty(1, 2, 64, device="cuda", dtype=torch.bfloat16).expand(10, 2, 64))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,heads,dk,dv", [([200], (64, 1, 1), 128, 128), ([130, 70], (24, 3, 3), 64, 128), ([1, 0, 90], (1, 30, 1), 32, 40),
                                                 ([600], (32, 1, 4), 64, 64)])
def test_many_heads_of_one_row(io, lengths, heads, dk, dv):
    """Few sequences whose heads share rows: workgroups of one row on several XCDs."""
    c = Case(lengths, heads, dk, dv, io, seed=60, state=True)
    _check_prefill(c, max_seqlen=max(lengths))
    _check_backward(c, max_seqlen=max(lengths))


@pytest.mark.parametrize("lengths", [[40, 30, 70], [400, 300, 700]])
def test_prefill_slots_without_a_state(lengths):
    """Slots of a batch that asks for no states: each sequence has its outputs
    whatever its slot's number, padding and repeated slots as ever."""
    from mamba_selective_ssm_ssd_amd import linear
    c = Case(lengths, (2, 2, 2), 64, 64, "bf16", seed=61)
    want, _ = linear.prefill(*c.args(), cu_seqlens=c.cu_dev, want_final=False)
    for slots, pool in (([7, 900, 3], None), ([2 ** 31 - 1, 0, 5], None), ([8, 0, 3], 9)):
        o = torch.full_like(want, 7.0)
        final = None if pool is None else torch.full((pool, 2, 64, 64), 5.0, device="cuda")
        linear.prefill(*c.args(), final=final, cu_seqlens=c.cu_dev, want_final=False, o=o,
                       slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
        assert torch.equal(o, want) and (final is None or (final == 5).all())
    o = torch.full_like(want, 7.0)
    linear.prefill(*c.args(), cu_seqlens=c.cu_dev, want_final=False, o=o, slots=torch.tensor([-3, 40, 40], dtype=torch.int32, device="cuda"))
    a, b = c.cu[1], c.cu[2]
    assert (o[:a] == 7).all() and torch.equal(o[a:b], want[a:b]) and torch.isnan(o[b:].float()).all()


INF_DECAYS = [0.0, -1e-6, -0.01, -0.3, -0.6]


def _infinite(state):
    """The same states with an infinity of each sign in column 5 of every head, and where they are."""
    s = state.clone()
    s[:, :, 3, 5], s[:, :, 9, 5] = float("inf"), float("-inf")
    at = torch.zeros_like(s, dtype=torch.bool)
    at[:, :, 3, 5] = at[:, :, 9, 5] = True
    return s, at


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("sd", ["f32", "bf16"])
def test_step_keeps_infinite_states(io, sd):
    """exp(log_decay) inf is inf, without any decay too; nothing else moves."""
    from mamba_selective_ssm_ssd_amd import linear
    c = Case([1] * 3, (5, 5, 5), 32, 40, io, seed=62)
    c.ld[:] = torch.tensor(INF_DECAYS)
    s0 = torch.randn(3, 5, 32, 40, device="cuda").to(DT[sd])
    s1, at = _infinite(s0)
    o0 = linear.decode_step(*c.args(), s0)
    o1 = linear.decode_step(*c.args(), s1)
    assert torch.equal(s1[~at], s0[~at])
    assert (s1[:, :, 3, 5] == float("inf")).all() and (s1[:, :, 9, 5] == float("-inf")).all()
    keep = torch.arange(40, device="cuda") != 5
    assert torch.equal(o1[..., keep], o0[..., keep])
    # q[3] inf - q[9] inf: an infinity where their signs differ
    a, b = c.q[..., 3].float(), c.q[..., 9].float()
    want = a * float("inf") + b * float("-inf")
    got, nan = o1[..., 5].float(), torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [40, 700, 2600])
def test_prompt_keeps_infinite_states(io, n):
    """The same of whole sequences, of a few segments folded and of many joined."""
    from mamba_selective_ssm_ssd_amd import capi, linear
    c = Case([n], (5, 5, 5), 32, 40, io, seed=63, state=True)
    # decays that leave more than nothing behind the prompt
    c.ld[:] = torch.tensor([0.0, -1e-6, -1e-4, -1e-3, -0.01])
    rc, seg, _ = capi.m3_linear_plan(linear.make_shape(1, n, 5, 5, 5, 32, 40, c.dt))
    assert rc == 0 and (seg == 0 if n == 40 else n <= 4 * seg if n == 700 and io == "bf16" else n > 4 * seg)
    o0, f0 = _run_prefill(c)
    c.state, at = _infinite(c.state)
    o1, f1 = _run_prefill(c)
    assert torch.equal(f1[~at], f0[~at])
    assert (f1[:, :, 3, 5] == float("inf")).all() and (f1[:, :, 9, 5] == float("-inf")).all()
    keep = torch.arange(40, device="cuda") != 5
    assert torch.equal(o1[..., keep], o0[..., keep]) and not torch.isfinite(o1[..., 5].float()).any()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 64), (128, 128), (64, 128)])
@pytest.mark.parametrize("lengths", [[150, 3], [900, 200]])
def test_outputs_do_not_depend_on_the_final_state(lengths, dk, dv, io):
    """Bit for bit: with the final state, without it, and in place."""
    from mamba_selective_ssm_ssd_amd import linear
    c = Case(lengths, (3, 3, 3), dk, dv, io, seed=64, state=True)
    o0, _ = _run_prefill(c)
    o1, none = linear.prefill(*c.args(), state=c.state, cu_seqlens=c.cu_dev, want_final=False)
    o2, _ = linear.prefill(*c.args(), state=c.state.clone(), cu_seqlens=c.cu_dev)
    assert none is None and torch.equal(o0, o1) and torch.equal(o0, o2)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(32, 40), (128, 128)])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("long", [[257, 256, 513], [1500], [129, 128, 300, 700, 256, 257]])
def test_many_short_sequences_and_a_few_cut_ones(long, state, dk, dv, io):
    """More sequences than segments of tokens: states are kept for the cut ones
    alone, whichever they are, in a workspace of garbage."""
    from mamba_selective_ssm_ssd_amd import capi, linear
    r = np.random.RandomState(len(long))
    lengths = [int(n) for n in r.permutation([0, 0, 1, *r.randint(1, 30, 40), *long])]
    c = Case(lengths, (2, 1, 2), dk, dv, io, seed=65, state=state)
    T, B = sum(lengths), len(lengths)
    for back in (False, True):
        ws = torch.full((linear.workspace_bytes(c.q, c.k, c.v, c.cu_dev, backward=back),), 255, dtype=torch.uint8, device="cuda")
        L = capi.m3_linear_plan(linear.make_shape(B, T, 2, 1, 2, dk, dv, c.dt))[1 + back]
        assert 0 < L < max(lengths) and T // L < B
        (_check_backward if back else _check_prefill)(c, workspace=ws)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0])
@pytest.mark.parametrize("lengths", [[70, 1, 0, 33], [700, 300], [1500]])
def test_scale(lengths, scale, io):
    """A factor of its own through the prompt, its gradients (the states' among
    them) and the step, of whole sequences, few segments and many."""
    from mamba_selective_ssm_ssd_amd import linear
    c = Case(lengths, (4, 2, 2), 64, 32, io, seed=66, state=True)
    final = torch.empty_like(c.state)
    o, _ = linear.prefill(*c.args(), state=c.state, final=final, cu_seqlens=c.cu_dev, scale=scale)
    wo, wf = ol.prefill(*c.host(), c.cu, _np(c.state), scale)
    ao, af = ol.prefill(*c.host(True), c.cu, np.abs(_np(c.state)), abs(scale))
    _check("o", o, wo, ao, c.dt)
    _check("final", final, wf, af, torch.float32)
    g = linear.backward(*c.args(), c.go, state=c.state, gfinal=c.gfinal, cu_seqlens=c.cu_dev, scale=scale)
    want = ol.backward(*c.host(), _np(c.go), c.cu, _np(c.state), _np(c.gfinal), scale)
    size = ol.backward(*c.host(True), np.abs(_np(c.go)), c.cu, np.abs(_np(c.state)), np.abs(_np(c.gfinal)), abs(scale))
    for n, w, a in zip(("q", "k", "v", "state"), want, size):
        _check("d" + n, g[n], w, a, c.dt if n != "state" else torch.float32)
    d = Case([1, 1], (4, 2, 2), 64, 32, io, seed=67, state=True)
    pool = d.state.clone()
    got = linear.decode_step(*d.args(), pool, scale=scale)
    wo, wf = ol.prefill(*d.host(), d.cu, _np(d.state), scale)
    ao, af = ol.prefill(*d.host(True), d.cu, np.abs(_np(d.state)), abs(scale))
    assert (np.abs(_np(got) - wo) <= U32 * ao + (1.01 * U16 * np.abs(wo) if io == "bf16" else 0)).all()
    _check("state", pool, wf, af, torch.float32)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 96), (24, 64)])
@pytest.mark.parametrize("lengths", [[70, 1, 0, 33], [700, 0, 300], [1500]])
def test_backward_from_bf16_states(lengths, dk, dv, io):
    """Initial states in bf16, of whole sequences, few segments and many: the gradient of one is fp32."""
    _check_backward(Case(lengths, (2, 2, 1), dk, dv, io, seed=68, state=True, sd=torch.bfloat16))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("B,T,heads", [(3, 90, (4, 2, 4)), (5, 1, (2, 2, 2)), (2, 700, (2, 1, 1)), (4, 64, (1, 3, 3))])
def test_backward_of_dense_batches(B, T, heads, state, io):
    """[B,T,H,D] rows without cu_seqlens, and the same with it: bit for bit."""
    from mamba_selective_ssm_ssd_amd import linear
    c = Case([T] * B, heads, 64, 32, io, seed=69, state=state)
    dense = [t.view(B, T, *t.shape[1:]) for t in (c.q, c.k, c.v, c.go)]
    g = linear.backward(*dense[:3], c.ld, dense[3], state=c.state, gfinal=c.gfinal)
    assert all(g[n].shape == dense["qkv".index(n)].shape for n in "qkv")
    flat = {n: t if n == "state" else t.flatten(0, 1) for n, t in g.items()}
    _compare_backward(c, flat)
    same = linear.backward(*c.args(), c.go, state=c.state, gfinal=c.gfinal, cu_seqlens=c.cu_dev, max_seqlen=T)
    assert all(torch.equal(flat[n], same[n]) for n in same)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_a_decay_that_is_nan_shows(io):
    """Heads whose log_decay is NaN have NaN for states and outputs, in the step,
    and in whole, folded and joined prompts; the others do not."""
    from mamba_selective_ssm_ssd_amd import linear
    nan = torch.tensor([False, True, False], device="cuda")
    c = Case([1] * 3, (3, 3, 3), 32, 40, io, seed=70, state=True)
    c.ld[nan] = float("nan")
    pool = c.state.clone()
    o = linear.decode_step(*c.args(), pool)
    assert torch.isnan(o[:, nan].float()).all() and torch.isfinite(o[:, ~nan].float()).all()
    assert torch.isnan(pool[:, nan]).all() and torch.isfinite(pool[:, ~nan]).all()
    for n in (100, 700, 2600):
        c = Case([n], (3, 3, 3), 32, 40, io, seed=71, state=True)
        c.ld[nan] = float("nan")
        o, f = _run_prefill(c)
        assert torch.isnan(f[:, nan]).all() and torch.isfinite(f[:, ~nan]).all()
        assert torch.isnan(o[1:, nan].float()).all() and torch.isfinite(o[:, ~nan].float()).all()
        g = _run_backward(c)
        assert torch.isnan(g["state"][:, nan]).all() and all(torch.isfinite(g[x][:, ~nan].float()).all() for x in g)
