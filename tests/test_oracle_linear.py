"""The fp64 oracle of linear attention and of the rotary norm (oracle/linear.py)
against forms it does not use: the masked quadratic form, differences for the
gradients, complex rotation."""
import numpy as np
import pytest

from oracle import linear as ol

CU = [0, 3, 3, 4, 11]


def _draw(seed, heads=(4, 2, 1), dk=3, dv=5, T=11):
    r = np.random.default_rng(seed)
    H = max(heads)
    return (*(r.standard_normal((T, h, d)) for h, d in zip(heads, (dk, dk, dv))), -r.uniform(0.01, 1.0, H),
            r.standard_normal((len(CU) - 1, H, dk, dv)), r)


def test_prefill_is_the_masked_product():
    q, k, v, ld, S0, _ = _draw(0)
    o, final = ol.prefill(q, k, v, ld, CU, S0, scale=0.7)
    for b, (lo, hi) in enumerate(zip(CU, CU[1:])):
        i = np.arange(hi - lo)
        for h in range(4):
            L = np.where(i[:, None] >= i, np.exp(ld[h] * (i[:, None] - i)), 0.0)
            qq, kk, vv = q[lo:hi, h], k[lo:hi, h // 2], v[lo:hi, 0]
            want = 0.7 * ((qq @ kk.T * L) @ vv + np.exp(ld[h] * (i + 1))[:, None] * (qq @ S0[b, h]))
            assert np.allclose(o[lo:hi, h], want, rtol=1e-12, atol=1e-12)
            n = hi - lo
            S = np.exp(ld[h] * n) * S0[b, h] + (kk * np.exp(ld[h] * (n - 1 - i))[:, None]).T @ vv
            assert np.allclose(final[b, h], S, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("heads", [(4, 2, 1), (1, 1, 3), (2, 2, 2)])
def test_backward_against_differences(heads):
    q, k, v, ld, S0, r = _draw(1, heads)
    go, gf = r.standard_normal((11, max(heads), 5)), r.standard_normal(S0.shape)

    def loss(q, k, v, S0):
        o, f = ol.prefill(q, k, v, ld, CU, S0)
        return np.sum(o * go) + np.sum(f * gf)

    args = [q, k, v, S0]
    grads = ol.backward(q, k, v, ld, go, CU, S0, gf)
    for i, (x, g) in enumerate(zip(args, grads)):
        d = r.standard_normal(x.shape)
        up, down = list(args), list(args)
        up[i], down[i] = x + 1e-5 * d, x - 1e-5 * d
        assert np.isclose((loss(*up) - loss(*down)) / 2e-5, np.sum(g * d), rtol=1e-7, atol=1e-7)


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rotate_is_a_complex_turn_and_its_gradient_matches_differences(halves, norm):
    r = np.random.default_rng(2)
    x, g, w = r.standard_normal((7, 2, 12)), r.standard_normal((7, 2, 12)), r.uniform(0.5, 1.5, 12)
    pos, f = r.integers(0, 1000, (2, 7)), r.uniform(0, 1, (2, 4))
    w = w if norm else None
    y = ol.norm_rotate(x, pos, f, w, norm, 1e-3, halves)
    n = x * (w / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-3)) if norm else x
    z = n[..., :4] + 1j * n[..., 4:8] if halves else n[..., 0:8:2] + 1j * n[..., 1:8:2]
    z = z * np.exp(1j * (pos.T @ f))[:, None]
    got = y[..., :4] + 1j * y[..., 4:8] if halves else y[..., 0:8:2] + 1j * y[..., 1:8:2]
    assert np.allclose(got, z, atol=1e-12) and np.allclose(y[..., 8:], n[..., 8:])
    dx, dw = ol.norm_rotate_backward(x, pos, f, g, w, norm, 1e-3, halves)
    loss = lambda x, w: np.sum(g * ol.norm_rotate(x, pos, f, w, norm, 1e-3, halves))  # noqa: E731
    d = r.standard_normal(x.shape)
    assert np.isclose((loss(x + 1e-5 * d, w) - loss(x - 1e-5 * d, w)) / 2e-5, np.sum(dx * d), rtol=1e-7)
    if norm:
        d = r.standard_normal(12)
        assert np.isclose((loss(x, w + 1e-5 * d) - loss(x, w - 1e-5 * d)) / 2e-5, np.sum(dw * d), rtol=1e-7)
