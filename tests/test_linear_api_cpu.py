"""Refusals, plans and workspace sizes of include/m3_linear.h and
include/m3_rotary.h.  Every call fails validation (or has nothing to do)
before any HIP call; pointers are never dereferenced."""
import ctypes

import pytest

from mamba_selective_ssm_ssd_amd import capi

FAKE, OFF = 0x10000, 0x10008
I, U, W, OK = capi.M3_ERR_INVALID_ARGUMENT, capi.M3_ERR_UNSUPPORTED, capi.M3_ERR_WORKSPACE, capi.M3_OK


def _lshape(**kw):
    d = dict(batch=2, tokens=100, max_seqlen=0, q_heads=4, k_heads=2, v_heads=1, key_dim=64, value_dim=32,
             io_dtype=capi.M3_DTYPE_BF16, state_dtype=capi.M3_DTYPE_F32, scale=1.0)
    return capi.m3_linear_shape_t(**{**d, **kw})


def _rows(h, d, data=FAKE, **kw):
    return capi.m3_rows_t(**{**dict(data=data, token_stride=h * d, head_stride=d), **kw})


def _prefill(shape=None, cu=FAKE, ws=FAKE, wn=1 << 40, ld=FAKE, slots=None, n=2, init=None, fin=FAKE, **rows):
    r = dict(q=_rows(4, 64), k=_rows(2, 64), v=_rows(1, 32), o=_rows(4, 32)) | rows
    return capi.m3_linear_prefill(shape or _lshape(), r["q"], r["k"], r["v"], ld, cu, slots, n, init, fin, r["o"], ws, wn, None)


def _decode(shape=None, ld=FAKE, slots=None, n=2, state=FAKE, **rows):
    r = dict(q=_rows(4, 64), k=_rows(2, 64), v=_rows(1, 32), o=_rows(4, 32)) | rows
    return capi.m3_linear_decode_step(shape or _lshape(), r["q"], r["k"], r["v"], ld, slots, n, state, r["o"], None)


def _backward(shape=None, cu=FAKE, ws=FAKE, wn=1 << 40, ld=FAKE, init=None, gfinal=None, ginit=None, **rows):
    r = dict(q=_rows(4, 64), k=_rows(2, 64), v=_rows(1, 32), go=_rows(4, 32), gq=_rows(4, 64), gk=_rows(2, 64), gv=_rows(1, 32)) | rows
    return capi.m3_linear_prefill_backward(shape or _lshape(), r["q"], r["k"], r["v"], ld, cu, init, r["go"], gfinal, r["gq"], r["gk"],
                                           r["gv"], ginit, ws, wn, None)


CALLS = {"prefill": _prefill, "decode": _decode, "backward": _backward}


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("field,value,expect", [
    ("batch", 0, I), ("q_heads", 0, I), ("k_heads", 3, I), ("v_heads", 3, I), ("key_dim", 0, I), ("value_dim", -8, I),
    ("key_dim", 60, U), ("value_dim", 136, U), ("key_dim", 256, U), ("io_dtype", 2, I), ("state_dtype", 7, I)])
def test_linear_shape_errors(call, field, value, expect):
    assert CALLS[call](_lshape(**{field: value})) == expect
    if call != "decode":
        size = capi.m3_linear_prefill_workspace_bytes if call == "prefill" else capi.m3_linear_prefill_backward_workspace_bytes
        assert size(_lshape(**{field: value})) == 0 and size(_lshape()) >= 256


def test_linear_length_errors():
    for call in (_prefill, _backward):
        assert call(_lshape(tokens=-1)) == I and call(_lshape(max_seqlen=-1)) == I
        assert call(_lshape(tokens=101), cu=None) == I                # equal sequences must divide the tokens
        assert call(_lshape(tokens=1 << 31)) == U


def test_more_than_one_launch_takes():
    # 2^32 threads: 256 x (3 scans x 2 column tiles) for each segment slot and head
    one = dict(q_heads=1, k_heads=1, v_heads=1)
    size = capi.m3_linear_prefill_workspace_bytes
    assert size(_lshape(batch=2795682, tokens=0, **one)) > 0 and size(_lshape(batch=2795683, tokens=0, **one)) == 0
    assert size(_lshape(batch=1, tokens=(1 << 31) - 1, **one)) > 0
    assert size(_lshape(batch=1, tokens=(1 << 31) - 1, q_heads=2, k_heads=1, v_heads=1)) == 0
    assert _prefill(_lshape(batch=2795683, tokens=0, **one)) == U and _backward(_lshape(batch=2795683, tokens=0, **one)) == U
    # the slots that a plan may use stay within what is counted
    for batch, tokens, heads in ((1, 256, 1000), (1, 4096, 32), (3, 300000, 1), (1, 520, 252), (40, 131072, 1), (1, 262144, 1)):
        s = _lshape(batch=batch, tokens=tokens, q_heads=heads, k_heads=heads, v_heads=heads)
        for L in capi.m3_linear_plan(s)[1:]:
            assert ((tokens // L if L else 0) + batch) * heads <= (batch + 8 + tokens / 1024) * heads + 512
    assert _decode(_lshape(batch=8388088, **one), n=1 << 23) == U
    # a wave of 64 for each token's q and k
    size = capi.m3_norm_rotate_backward_workspace_bytes
    assert size(_rshape(tokens=33554429, q_heads=1, k_heads=1)) > 0 and size(_rshape(tokens=33554430, q_heads=1, k_heads=1)) == 0
    assert size(_rshape(tokens=33554429, q_heads=33, k_heads=1)) == 0          # two waves of q


@pytest.mark.parametrize("call,names", [("prefill", "qkvo"), ("decode", "qkvo"), ("backward", ("q", "k", "v", "go", "gq", "gk", "gv"))])
def test_linear_row_errors(call, names):
    f = CALLS[call]
    for n in names:
        h, d = (4 if n in ("q", "o", "go", "gq") else 2 if "k" in n else 1), (64 if n[-1] in "qk" else 32)
        for bad in (dict(data=None), dict(data=OFF), dict(token_stride=h * d + 4), dict(head_stride=d + 1), dict(token_stride=-h * d),
                    dict(token_stride=1 << 24), dict(head_stride=1 << 40)):
            assert f(**{n: _rows(h, d, **bad)}) == I, (n, bad)
        assert f(**{n: None}) == I
    for n in ("o",) if call != "backward" else ("gq",):               # outputs that overlap themselves
        d = 32 if n == "o" else 64
        for bad in (dict(token_stride=0), dict(head_stride=0), dict(head_stride=d - 8), dict(token_stride=4 * d - 8)):
            assert f(**{n: _rows(4, d, **bad)}) == I, bad


def test_linear_pointer_and_workspace_errors():
    for call in (_prefill, _decode, _backward):
        assert call(ld=None) == I and call(ld=FAKE + 2) == I
    for call in (_prefill, _backward):
        assert call(cu=FAKE + 2) == I and call(init=OFF) == I
        assert call(ws=None) == W and call(ws=OFF) == W and call(wn=255) == W
    assert _prefill(slots=FAKE + 1) == I and _prefill(n=1) == I and _prefill(n=-1, slots=FAKE) == I and _prefill(fin=OFF) == I
    assert _decode(slots=FAKE + 1) == I and _decode(n=1) == I and _decode(state=None) == I and _decode(state=OFF) == I
    assert _backward(gfinal=OFF) == I and _backward(ginit=OFF) == I
    assert capi.m3_linear_prefill(None, *[None] * 5, None, 0, None, None, None, None, 0, None) == I


def test_linear_plan_and_workspace():
    # a short prompt is not cut
    assert capi.m3_linear_plan(_lshape(batch=1, tokens=200)) == (OK, 0, 0)
    assert capi.m3_linear_prefill_workspace_bytes(_lshape(batch=1, tokens=200)) == 256
    # nor are enough like sequences to fill the chip, nor sequences that max_seqlen says are short
    assert capi.m3_linear_plan(_lshape(batch=256, tokens=256 * 2048, max_seqlen=2048)) == (OK, 0, 0)
    assert capi.m3_linear_plan(_lshape(batch=256, tokens=256 * 2048))[1] > 0
    assert capi.m3_linear_plan(_lshape(batch=100, tokens=20000, max_seqlen=200))[1] == 0
    # a long one is; slots of an fp32 state for every segment and sequence
    for heads, T in ((1, 100000), (8, 65536), (4, 5000)):
        s = _lshape(batch=3, tokens=T, q_heads=heads, k_heads=heads, v_heads=heads, key_dim=128, value_dim=128)
        rc, a, b = capi.m3_linear_plan(s)
        assert rc == OK and a % 64 == b % 64 == 0 and 0 < a < T and 0 < b < T
        need = (T // a + 3) * heads * 128 * 128 * 4
        assert need <= capi.m3_linear_prefill_workspace_bytes(s) < need + 256
        need = 2 * (T // b + 3) * heads * 128 * 128 * 4
        assert need <= capi.m3_linear_prefill_backward_workspace_bytes(s) < need + 512
    # fp32 parts of the gradients of shared rows
    s = _lshape(batch=1, tokens=200)
    need = 200 * 4 * (64 + 32) * 4                                    # k and v; q has a row per head
    assert need <= capi.m3_linear_prefill_backward_workspace_bytes(s) <= need + 512
    assert capi.m3_linear_plan(_lshape(batch=0))[0] == I


def test_outputs_that_start_in_another_operand():
    at = lambda h, d, n: _rows(h, d, data=n << 20)  # noqa: E731
    fine = dict(q=at(4, 64, 1), k=at(2, 64, 2), v=at(1, 32, 3))
    for n in "qkv":
        assert _prefill(**fine, o=at(4, 32, "?qkv".index(n))) == I and _decode(**fine, o=at(4, 32, "?qkv".index(n))) == I
    grads = dict(go=at(4, 32, 4), gq=at(4, 64, 5), gk=at(2, 64, 6), gv=at(1, 32, 7))
    for n, (h, d) in dict(gq=(4, 64), gk=(2, 64), gv=(1, 32)).items():
        for other in (1, 2, 3, 4, 5, 6, 7):
            if other != list(grads).index(n) + 4:
                assert _backward(**fine, **{**grads, n: at(h, d, other)}) == I, (n, other)
    assert _backward(**fine, **grads, gfinal=FAKE, ginit=FAKE) == I and _backward(**fine, **grads, init=FAKE, ginit=FAKE) == I
    # the heads' parts of one token beyond what a chunk's offsets count
    big = _lshape(batch=1, tokens=1, q_heads=1 << 18, k_heads=1, v_heads=1)
    assert _prefill(big) == U and capi.m3_linear_prefill_backward_workspace_bytes(big) == 0


def _rshape(**kw):
    d = dict(tokens=10, q_heads=4, k_heads=2, dim=64, rot=32, axes=1, io_dtype=capi.M3_DTYPE_BF16, pos_int64=0, halves=0, norm=1, eps=1e-6)
    return capi.m3_rotary_shape_t(**{**d, **kw})


def _rotate(shape=None, pos=FAKE, freq=FAKE, qw=FAKE, kw=FAKE, **rows):
    r = dict(q=_rows(4, 64), k=_rows(2, 64), qo=_rows(4, 64), ko=_rows(2, 64)) | rows
    return capi.m3_norm_rotate(shape or _rshape(), r["q"], r["k"], pos, freq, qw, kw, r["qo"], r["ko"], None)


def _rotate_back(shape=None, pos=FAKE, freq=FAKE, qw=FAKE, kw=FAKE, dqw=FAKE, dkw=FAKE, ws=FAKE, wn=1 << 40, **rows):
    r = dict(q=_rows(4, 64), k=_rows(2, 64), gq=_rows(4, 64), gk=_rows(2, 64), qo=_rows(4, 64), ko=_rows(2, 64)) | rows
    return capi.m3_norm_rotate_backward(shape or _rshape(), r["q"], r["k"], pos, freq, qw, kw, r["gq"], r["gk"], r["qo"], r["ko"], dqw, dkw,
                                        ws, wn, None)


@pytest.mark.parametrize("call", [_rotate, _rotate_back])
def test_rotary_errors(call):
    for field, value, expect in (("tokens", -1, I), ("q_heads", 0, I), ("k_heads", -1, I), ("dim", 0, I), ("rot", 72, I), ("rot", 0, I),
                                 ("axes", 0, I), ("io_dtype", 5, I), ("eps", -1.0, I), ("eps", float("nan"), I), ("dim", 60, U), ("dim", 264, U),
                                 ("rot", 12, U), ("axes", 5, U), ("tokens", 1 << 40, U)):
        assert call(_rshape(**{field: value})) == expect, (field, value)
        assert capi.m3_norm_rotate_backward_workspace_bytes(_rshape(**{field: value})) == 0
    assert call(pos=None) == I and call(pos=FAKE + 2) == I and call(_rshape(pos_int64=1), pos=FAKE + 4) == I
    assert call(freq=None) == I and call(freq=OFF) == I and call(qw=OFF) == I and call(kw=OFF) == I
    assert call(_rshape(norm=0)) == I                                 # weights without their norm
    for n, h in (("q", 4), ("k", 2), ("qo", 4), ("ko", 2)):
        for bad in (dict(data=None), dict(data=OFF), dict(token_stride=h * 64 + 4), dict(head_stride=65), dict(head_stride=-64)):
            assert call(**{n: _rows(h, 64, **bad)}) == I, (n, bad)
        assert call(**{n: None}) == I
    for n, h in (("qo", 4), ("ko", 2)):
        for bad in (dict(token_stride=0), dict(head_stride=0), dict(head_stride=56)):
            assert call(**{n: _rows(h, 64, **bad)}) == I, (n, bad)


def test_rotary_backward_errors():
    assert _rotate_back(ws=None) == W and _rotate_back(ws=OFF) == W and _rotate_back(wn=16) == W
    assert _rotate_back(dqw=None) == I and _rotate_back(kw=None) == I and _rotate_back(dkw=FAKE + 2) == I
    assert _rotate_back(gq=_rows(4, 64, data=None)) == I and _rotate_back(gk=None) == I
    assert capi.m3_norm_rotate_backward_workspace_bytes(_rshape(tokens=0)) == 2 * 64 * 4


def test_rotary_outputs_that_start_in_another_operand():
    at = lambda h, n, **kw: _rows(h, 64, data=n << 20, **kw)  # noqa: E731
    fine = dict(q=at(4, 1), k=at(2, 2), qo=at(4, 3), ko=at(2, 4))
    bad = [dict(qo=at(4, 2)), dict(ko=at(2, 1)), dict(ko=at(2, 3)), dict(qo=at(4, 1, token_stride=512)), dict(ko=at(2, 2, head_stride=96, token_stride=192))]
    for b in bad:
        assert _rotate(**{**fine, **b}) == I, b
        assert _rotate_back(**{**fine, **b}, gq=at(4, 5), gk=at(2, 6)) == I, b
    for b in (dict(qo=at(4, 6)), dict(ko=at(2, 5)), dict(qo=at(4, 5, head_stride=128, token_stride=512))):
        assert _rotate_back(**{**fine, **b}, gq=at(4, 5), gk=at(2, 6)) == I, b


def test_rotary_nothing_to_do():
    assert _rotate(_rshape(tokens=0), pos=None) == OK


def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    from mamba_selective_ssm_ssd_amd import linear, rotary
    q = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        linear.prefill(q, q, q, torch.zeros(2))
    with pytest.raises(ValueError):
        linear.decode_step(q, q, q, torch.zeros(2), torch.zeros(4, 2, 64, 64))
    with pytest.raises(ValueError):
        linear.backward(q, q, q, torch.zeros(2), q)
    with pytest.raises(ValueError):
        rotary.norm_rotate(q, q, torch.zeros(4, dtype=torch.int32), torch.zeros(32))


def test_axes_table():
    torch = pytest.importorskip("torch")
    from mamba_selective_ssm_ssd_amd import rotary
    f = torch.arange(1.0, 7.0)
    t = rotary.axes_table(f, (2, 3, 1))
    assert torch.equal(t, torch.tensor([[1.0, 2, 0, 0, 0, 0], [0, 0, 3, 4, 5, 0], [0, 0, 0, 0, 0, 6]]))
    t = rotary.axes_table(f, (2, 3, 1), interleaved=True)
    assert torch.equal(t, torch.tensor([[1.0, 0, 0, 4, 0, 0], [0, 2, 0, 0, 5, 6], [0, 0, 3, 0, 0, 0]]))
    with pytest.raises(ValueError):
        rotary.axes_table(f, (2, 3))
    assert ctypes.sizeof(capi.m3_rows_t) == 24


def test_every_output_against_every_operand():
    def call(f, heads, addresses, **kw):
        return f(**kw, **{n: _rows(*heads[n], data=p) if n in heads else p for n, p in addresses.items()})

    h = dict(q=(4, 64), k=(2, 64), v=(1, 32), o=(4, 32), go=(4, 32), gq=(4, 64), gk=(2, 64), gv=(1, 32), qo=(4, 64), ko=(2, 64))
    r = {**h, "gq": (4, 64), "gk": (2, 64)}
    for f, heads, names, outputs, may in (
            (_prefill, h, "q k v o ld cu slots init fin ws", "o fin ws", {("fin", "init")}),
            (_decode, h, "q k v o ld slots state", "o state", set()),
            (_backward, h, "q k v go gq gk gv ld cu init gfinal ginit ws", "gq gk gv ginit ws", set()),
            (_rotate, r, "q k qo ko pos freq qw kw", "qo ko", {("qo", "q"), ("ko", "k")}),
            (_rotate_back, r, "q k gq gk qo ko pos freq qw kw dqw dkw ws", "qo ko dqw dkw ws",
             {("qo", "q"), ("qo", "gq"), ("ko", "k"), ("ko", "gk")})):
        names = names.split()
        at = {n: (i + 1) << 20 for i, n in enumerate(names)}
        for out in outputs.split():
            for other in names:
                if out != other and (out, other) not in may:
                    assert call(f, heads, {**at, out: at[other]}) == I, (f.__name__, out, other)


def test_operands_without_a_token_are_not_compared():
    # rows of no token may point anywhere; the other operands are compared all the same
    s = _rshape(tokens=0)
    assert _rotate(s, pos=None, qw=FAKE, kw=FAKE) == OK
    assert _rotate_back(s, dqw=2 * FAKE, dkw=2 * FAKE, ws=3 * FAKE) == I and _rotate_back(s, dqw=2 * FAKE, dkw=3 * FAKE, ws=3 * FAKE) == I


def test_workspace_of_many_sequences():
    """States of segments are kept for cut sequences: at most 2 tokens / L, however many sequences there are."""
    for batch, tokens, longest, heads in ((1000, 60000, 8192, 32), (256, 128000, 0, 64), (5000, 20000, 1000, 4), (300, 300 * 257, 0, 8),
                                          (7, 4999, 0, 32), (40, 9000, 8000, 2)):
        s = _lshape(batch=batch, tokens=tokens, max_seqlen=longest, q_heads=heads, k_heads=heads, v_heads=heads, key_dim=128, value_dim=128)
        rc, a, b = capi.m3_linear_plan(s)
        assert rc == OK and a > 0 and b > 0
        for L, n, size in ((a, 1, capi.m3_linear_prefill_workspace_bytes), (b, 2, capi.m3_linear_prefill_backward_workspace_bytes)):
            states = min(tokens // L + batch, max(2 * tokens // L, 1))
            assert size(s) <= n * (states * heads * 128 * 128 * 4 + 256), (batch, tokens, L)
