"""Norm of queries and keys with the position rotation on the GPU against the
fp64 oracle (oracle/linear.py), and its gradients.

Tolerances.  One result is a sum of two products of fp32 values with a sine and
a cosine that are off by at most 2^-22 (1.3e-7 from the hardware plus the
rounding of the angle's fraction of a turn, 2 pi 2^-25), after a norm of a few
steps of 2^-24: |error| <= 16 x 2^-24 (|n_u| + |n_v|) before the result is
rounded to its type (bf16: at most 2^-8 of it).  The gradient subtracts two
terms of that kind, each bounded by its own size: at most 64 x 2^-24 of their
sum.  A weight's gradient sums T x H products in fp32, at most 64 of them one
after the other in a lane and in pairs from there on: 128 x 2^-24 of the sum
of their sizes.
"""
import numpy as np
import pytest

from oracle import linear as ol

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _setup(T, hq, hk, D, rot, io, axes=1, fused=False, weight=True, far=False, pos64=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    if fused:
        rows = torch.randn(T, hq + hk + 2, D, generator=g).to(DT[io]).cuda()
        q, k = rows[:, :hq], rows[:, hq:hq + hk]
    else:
        q, k = (torch.randn(T, h, D, generator=g).to(DT[io]).cuda() for h in (hq, hk))
    n = rot // 2
    f = (10000.0 ** (-torch.arange(n) / n)).float()
    from mamba_selective_ssm_ssd_amd import rotary
    sections = [n // axes + (a < n % axes) for a in range(axes)]
    f = rotary.axes_table(f, sections, interleaved=bool(seed % 2)).cuda()
    pos = torch.randint(0, (1 << 40) if far and pos64 else (1 << 20) if far else 5000, (axes, T), generator=g)
    pos = pos.to(torch.int64 if pos64 else torch.int32).cuda()
    w = [1 + 0.25 * torch.randn(D, generator=g).cuda() if weight else None for _ in range(2)]
    return q, k, pos, f, *w


def _size(x, pos, f, w, norm, halves):
    """Size of the two terms of every result: |n_u| + |n_v|."""
    n = np.abs(ol.norm_rotate(x, np.zeros_like(pos), f, w, norm, 1e-6, halves))
    m, out = f.shape[1], n.copy()
    a, b = (slice(0, m), slice(m, 2 * m)) if halves else (slice(0, 2 * m, 2), slice(1, 2 * m, 2))
    out[..., a] += n[..., b]
    out[..., b] += n[..., a]
    return out


CASES = [
    # T, hq, hk, D, rot, axes, halves, norm, weight, far, pos64, fused
    (1, 1, 1, 8, 8, 1, False, True, True, False, False, False),
    (5, 16, 16, 64, 32, 1, False, True, True, True, True, False),
    (37, 5, 2, 128, 128, 1, True, True, True, False, False, True),
    (130, 32, 8, 128, 64, 1, True, True, False, True, False, True),
    (33, 3, 1, 96, 96, 3, True, True, True, False, False, False),
    (33, 3, 3, 80, 40, 2, False, False, False, True, True, True),
    (7, 64, 64, 16, 16, 1, False, True, True, False, False, False),
    (9, 7, 1, 256, 256, 4, True, True, True, True, False, False),
    (20, 40, 40, 32, 8, 1, True, False, False, False, False, False),
    (11, 2, 1, 200, 96, 2, False, True, True, True, True, False),
]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES)
def test_norm_rotate(case, io):
    from mamba_selective_ssm_ssd_amd import rotary
    T, hq, hk, D, rot, axes, halves, norm, weight, far, pos64, fused = case
    q, k, pos, f, qw, kw = _setup(T, hq, hk, D, rot, io, axes, fused, weight, far, pos64, seed=T)
    got = rotary.norm_rotate(q, k, pos, f, norm=norm, q_weight=qw, k_weight=kw, halves=halves)
    for x, w, y in ((q, qw, got[0]), (k, kw, got[1])):
        want = ol.norm_rotate(_np(x), _np(pos), _np(f), _np(w), norm, 1e-6, halves)
        tol = 16 * E * _size(_np(x), _np(pos), _np(f), _np(w), norm, halves)
        tol += 1.01 * 2.0 ** -8 * np.abs(want) if io == "bf16" else 0
        err = np.abs(_np(y) - want)
        print(f"worst {float((err / tol).max()):.3f} of the bound", flush=True)
        assert y.dtype == x.dtype
        assert bool((err <= tol).all())


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES + [(2500, 3, 2, 64, 64, 1, True, True, True, False, False, False)])
def test_norm_rotate_backward(case, io):
    from mamba_selective_ssm_ssd_amd import rotary
    T, hq, hk, D, rot, axes, halves, norm, weight, far, pos64, fused = case
    q, k, pos, f, qw, kw = _setup(T, hq, hk, D, rot, io, axes, fused, weight, far, pos64, seed=T)
    gq, gk = (torch.randn(x.shape, generator=torch.Generator().manual_seed(i)).to(DT[io]).cuda() for i, x in enumerate((q, k)))
    got = rotary.norm_rotate_backward(q, k, pos, f, gq, gk, norm=norm, q_weight=qw, k_weight=kw, halves=halves)
    assert set(got) == {"q", "k"} | ({"q_weight", "k_weight"} if weight else set())
    for n, x, g, w in (("q", q, gq, qw), ("k", k, gk, kw)):
        dx, dw = ol.norm_rotate_backward(_np(x), _np(pos), _np(f), _np(g), _np(w), norm, 1e-6, halves)
        gn = _size(_np(g), _np(pos), _np(f), None, False, halves)
        a, r, size = np.abs(_np(x)), 1.0, gn
        if norm:
            r = 1 / np.sqrt(np.mean(a * a, -1, keepdims=True) + 1e-6)
            wg = gn * (np.abs(_np(w)) if weight else 1)
            size = r * wg + r ** 3 * a * np.mean(a * wg, -1, keepdims=True)
        tol = 64 * E * size + (1.01 * 2.0 ** -8 * np.abs(dx) if io == "bf16" else 0)
        err = np.abs(_np(got[n]) - dx)
        print(f"d{n}: worst {float((err / tol).max()):.3f} of the bound", flush=True)
        assert got[n].dtype == x.dtype
        assert bool((err <= tol).all())
        if weight:
            tol = 128 * E * np.sum(gn * a * r, axis=(0, 1))
            err = np.abs(_np(got[n + "_weight"]) - dw)
            print(f"d{n}_weight: worst {float((err / tol).max()):.3f} of the bound", flush=True)
            assert bool((err <= tol).all())


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("case", [
    # rows enough that a wave takes several sets of one token, the last of them in part
    (1100, 37, 3, 128, 128, 1, True, True, True, False, False, False),
    (1100, 20, 20, 64, 32, 1, False, True, True, True, False, True),
    (1100, 70, 1, 8, 8, 1, False, True, False, False, False, False),
    (1100, 5, 2, 256, 128, 2, True, False, False, False, True, False)])
def test_norm_rotate_many_rows(case, io):
    test_norm_rotate(case, io)


def test_heads_outside_tokens_and_no_keys():
    """Rows as [head][token][channel], broadcast inputs, and queries alone."""
    from mamba_selective_ssm_ssd_amd import rotary
    q, k, pos, f, qw, kw = _setup(50, 4, 2, 64, 64, "bf16")
    want = rotary.norm_rotate(q, k, pos, f, q_weight=qw, k_weight=kw)
    turned = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k)]
    outs = [torch.empty(h, 50, 64, device="cuda", dtype=q.dtype).transpose(0, 1) for h in (4, 2)]
    rotary.norm_rotate(*turned, pos, f, q_weight=qw, k_weight=kw, q_out=outs[0], k_out=outs[1])
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    one = rotary.norm_rotate(q[:, :1].expand(50, 4, 64), k[:1].expand(50, 2, 64), pos, f)
    full = rotary.norm_rotate(q[:, :1].repeat(1, 4, 1), k[:1].repeat(50, 1, 1), pos, f)
    assert all(torch.equal(a, b) for a, b in zip(one, full))
    y, none = rotary.norm_rotate(q, k[:, :0], pos, f, q_weight=qw)
    assert torch.equal(y, want[0]) and none.shape == (50, 0, 64)
    g = rotary.norm_rotate_backward(q, k[:, :0], pos, f, q, k[:, :0], q_weight=qw)
    ref = rotary.norm_rotate_backward(q, k, pos, f, q, k, q_weight=qw, k_weight=kw)
    assert torch.equal(g["q"], ref["q"]) and g["k"].shape == (50, 0, 64)


def test_in_place_batches_and_far_rows():
    from mamba_selective_ssm_ssd_amd import rotary
    q, k, pos, f, qw, kw = _setup(60, 4, 2, 64, 64, "bf16")
    want = rotary.norm_rotate(q, k, pos, f, q_weight=qw, k_weight=kw)
    batch = rotary.norm_rotate(q.view(3, 20, 4, 64), k.view(3, 20, 2, 64), pos, f, q_weight=qw, k_weight=kw)
    assert all(torch.equal(a, b.flatten(0, 1)) for a, b in zip(want, batch))
    rows = torch.cat([q, k, q], dim=1)
    q2, k2 = rows[:, :4], rows[:, 4:6]
    rotary.norm_rotate(q2, k2, pos, f, q_weight=qw, k_weight=kw, q_out=q2, k_out=k2)
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1]) and torch.equal(rows[:, 6:], q)


def test_empty_and_zero_rows():
    from mamba_selective_ssm_ssd_amd import rotary
    q, k, pos, f, qw, kw = _setup(4, 2, 1, 64, 64, "bf16")
    e = rotary.norm_rotate(q[:0], k[:0], pos[:, :0].contiguous(), f, q_weight=qw, k_weight=kw)
    assert e[0].shape == (0, 2, 64)
    g = rotary.norm_rotate_backward(q[:0], k[:0], pos[:, :0].contiguous(), f, q[:0], k[:0], q_weight=qw, k_weight=kw)
    assert not g["q_weight"].any() and not g["k_weight"].any()
    y, _ = rotary.norm_rotate(torch.zeros_like(q), k, pos, f, q_weight=qw, k_weight=kw)
    assert not y.any()
    # a non-finite row stays by itself
    q0 = rotary.norm_rotate(q, k, pos, f, q_weight=qw, k_weight=kw)[0]
    q[2, 1, 3] = float("nan")
    q1 = rotary.norm_rotate(q, k, pos, f, q_weight=qw, k_weight=kw)[0]
    keep = torch.ones(4, 2, dtype=torch.bool)
    keep[2, 1] = False
    assert torch.equal(q0[keep], q1[keep]) and torch.isnan(q1[2, 1].float()).all()


def test_refusals():
    from mamba_selective_ssm_ssd_amd import capi, rotary
    q, k, pos, f, qw, kw = _setup(4, 2, 1, 64, 64, "bf16")
    with pytest.raises(capi.M3Error):                                    # a weight without its norm
        rotary.norm_rotate(q, k, pos, f, norm=False, q_weight=qw)
    with pytest.raises(capi.M3Error):                                    # pairs that do not fill eight channels
        rotary.norm_rotate(q, k, pos, f[:, :30].contiguous())
    with pytest.raises(capi.M3Error):
        rotary.norm_rotate(q, k, pos, torch.zeros(1, 36, device="cuda"))
    with pytest.raises(capi.M3Error):
        rotary.norm_rotate(q, k, pos, f, eps=-1.0)
    with pytest.raises(capi.M3Error):
        rotary.norm_rotate_backward(q, k, pos, f, q, k, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    for bad in (dict(positions=pos[:, :3].contiguous()), dict(positions=pos.float()), dict(q_weight=qw[:32]), dict(q_weight=qw.bfloat16()),
                dict(k=k.float()), dict(k=k[:3]), dict(inv_freq=f.double()), dict(q_out=q[:3])):
        a = dict(q=q, k=k, positions=pos, inv_freq=f) | bad
        with pytest.raises(ValueError):
            rotary.norm_rotate(a.pop("q"), a.pop("k"), a.pop("positions"), a.pop("inv_freq"), **a)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("eps", [0.0, 1e-40])
@pytest.mark.parametrize("T,hq,hk,D,rot,halves", [(7, 5, 3, 64, 64, True), (40, 1, 2, 96, 48, False), (2500, 3, 9, 64, 32, True),
                                                 (9, 7, 1, 8, 8, False), (3, 3, 5, 256, 256, True)])
def test_norm_without_eps_and_sets_of_rows_in_part(T, hq, hk, D, rot, halves, eps, io):
    """No eps, and head counts that leave a wave's last set of rows in part: the
    places of no row must not reach the weights' gradients."""
    from mamba_selective_ssm_ssd_amd import rotary
    q, k, pos, f, qw, kw = _setup(T, hq, hk, D, rot, io, seed=D)
    gq, gk = (torch.randn(x.shape, generator=torch.Generator().manual_seed(i)).to(DT[io]).cuda() for i, x in enumerate((q, k)))
    y = rotary.norm_rotate(q, k, pos, f, eps=eps, q_weight=qw, k_weight=kw, halves=halves)
    got = rotary.norm_rotate_backward(q, k, pos, f, gq, gk, eps=eps, q_weight=qw, k_weight=kw, halves=halves)
    r16 = 1.01 * 2.0 ** -8 if io == "bf16" else 0
    for n, x, g, w, out in (("q", q, gq, qw, y[0]), ("k", k, gk, kw, y[1])):
        x, g, w = _np(x), _np(g), _np(w)
        want = ol.norm_rotate(x, _np(pos), _np(f), w, True, eps, halves)
        # rows of normal numbers: their mean of squares is far above eps, so _size's own eps changes nothing here
        assert np.mean(x * x, -1).min() > 1e-3
        assert (np.abs(_np(out) - want) <= 16 * E * 1.001 * _size(x, _np(pos), _np(f), w, True, halves) + r16 * np.abs(want)).all()
        dx, dw = ol.norm_rotate_backward(x, _np(pos), _np(f), g, w, True, eps, halves)
        gn, a = _size(g, _np(pos), _np(f), None, False, halves), np.abs(x)
        r = 1 / np.sqrt(np.mean(a * a, -1, keepdims=True) + eps)
        size = r * gn * np.abs(w) + r ** 3 * a * np.mean(a * gn * np.abs(w), -1, keepdims=True)
        assert (np.abs(_np(got[n]) - dx) <= 64 * E * size + r16 * np.abs(dx)).all()
        assert (np.abs(_np(got[n + "_weight"]) - dw) <= 128 * E * np.sum(gn * a * r, axis=(0, 1))).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("halves", [False, True])
def test_gradients_in_place(halves, norm, io):
    """Through the C ABI: the gradients of q and k in the rows of gq and gk, and in the rows of q and k."""
    from mamba_selective_ssm_ssd_amd import capi, rotary
    T, hq, hk, D = 70, 5, 3, 96
    q, k, pos, f, qw, kw = _setup(T, hq, hk, D, 64, io, weight=norm)
    gq, gk = (torch.randn(x.shape, generator=torch.Generator().manual_seed(i)).to(DT[io]).cuda() for i, x in enumerate((q, k)))
    want = rotary.norm_rotate_backward(q, k, pos, f, gq, gk, norm=norm, q_weight=qw, k_weight=kw, halves=halves)
    shape = capi.m3_rotary_shape_t(T, hq, hk, D, 64, 1, capi.M3_DTYPE_BF16 if io == "bf16" else capi.M3_DTYPE_F32, 0, halves, norm, 1e-6)
    ws = torch.empty(capi.m3_norm_rotate_backward_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    rows = lambda t: capi.m3_rows_t(t.data_ptr(), t.stride(0), t.stride(1))  # noqa: E731
    for over in ("g", "x"):
        x, g = [q.clone(), k.clone()], [gq.clone(), gk.clone()]
        out = g if over == "g" else x
        dw = [torch.empty(D, device="cuda") if norm else None for _ in range(2)]
        rc = capi.m3_norm_rotate_backward(shape, rows(x[0]), rows(x[1]), pos.data_ptr(), f.data_ptr(),
                                          *(t.data_ptr() if norm else None for t in (qw, kw)), rows(g[0]), rows(g[1]), rows(out[0]), rows(out[1]),
                                          *(t.data_ptr() if norm else None for t in dw), ws.data_ptr(), ws.numel(),
                                          torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        assert torch.equal(out[0], want["q"]) and torch.equal(out[1], want["k"])
        assert not norm or torch.equal(dw[0], want["q_weight"]) and torch.equal(dw[1], want["k_weight"])
