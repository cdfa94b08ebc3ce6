"""The oracle of the factor network's operators, pinned by what it does not compute by:
differences of the forward passes, the quadratic form of the attention, and the polynomial
on the singular values (float64, no GPU)."""
import numpy as np
import pytest

from oracle import factor_network as F


def _difference(fn, x, dx, h=1e-6):
    return (fn(x + h * dx) - fn(x - h * dx)) / (2 * h)


def test_layer_norm_rows_have_mean_zero_and_variance_one():
    x = np.random.default_rng(0).normal(3, 2, (5, 7))
    y, mean, rstd = F.layer_norm_fwd(x, eps=0.0)
    np.testing.assert_allclose(y.mean(-1), 0, atol=1e-14)
    np.testing.assert_allclose((y ** 2).mean(-1), 1, rtol=1e-14)
    np.testing.assert_allclose(y / rstd[:, None] + mean[:, None], x, rtol=1e-13)


def test_layer_norm_gradients_by_differences():
    rng = np.random.default_rng(1)
    x, dy, u = (rng.normal(size=(4, 9)) for _ in range(3))
    w, b, dw, db = (rng.normal(size=9) for _ in range(4))
    _, mean, rstd = F.layer_norm_fwd(x, w, b)
    gx, gw, gb = F.layer_norm_bwd(dy, x, w, mean, rstd)
    loss = lambda x_, w_, b_: (F.layer_norm_fwd(x_, w_, b_)[0] * dy).sum()  # noqa: E731
    np.testing.assert_allclose((gx * u).sum(), _difference(lambda z: loss(z, w, b), x, u), rtol=1e-7)
    np.testing.assert_allclose((gw * dw).sum(), _difference(lambda z: loss(x, z, b), w, dw), rtol=1e-7)
    np.testing.assert_allclose((gb * db).sum(), _difference(lambda z: loss(x, w, z), b, db), rtol=1e-7)


def _attention(seed, B=2, T=6, H=3, dk=4, dv=5):
    rng = np.random.default_rng(seed)
    q, k = (rng.normal(size=(B, T, H, dk)) for _ in range(2))
    v = rng.normal(size=(B, T, H, dv))
    return rng, q, k, v, np.array([-0.1, 0.0, -np.inf]), rng.normal(size=(B, H, dk, dv))


def test_attention_is_the_decayed_quadratic_form():
    _, q, k, v, g, S0 = _attention(2)
    o, S = F.linear_attention_fwd(q, k, v, g, 0.5, S0)
    T = q.shape[1]
    gap = np.arange(T)[:, None] - np.arange(T)
    with np.errstate(invalid="ignore"):
        L = np.where(gap > 0, np.exp(g[:, None, None] * np.maximum(gap, 1)), gap == 0)
    want = np.einsum("bthk,bshk,hts,bshv->bthv", q, k, L, v)
    first = np.exp(g[None, :] * np.arange(1, T + 1)[:, None])
    want += np.einsum("bthk,bhkv,th->bthv", q, S0, first)
    np.testing.assert_allclose(o, 0.5 * want, rtol=1e-12, atol=1e-13)
    # the state carries on: two halves equal the whole
    o1, mid = F.linear_attention_fwd(q[:, :4], k[:, :4], v[:, :4], g, 0.5, S0)
    o2, end = F.linear_attention_fwd(q[:, 4:], k[:, 4:], v[:, 4:], g, 0.5, mid)
    np.testing.assert_allclose(np.concatenate([o1, o2], 1), o, rtol=1e-12)
    np.testing.assert_allclose(end, S, rtol=1e-12)


@pytest.mark.parametrize("lengths", [None, [6, 3], [0, 1]])
def test_attention_gradients_by_differences(lengths):
    rng, q, k, v, g, S0 = _attention(3)
    n = None if lengths is None else np.array(lengths)
    do, dS = rng.normal(size=v.shape), rng.normal(size=S0.shape)
    grads = F.linear_attention_bwd(q, k, v, g, do, 0.7, S0, dS, n)

    def loss(*args):
        o, S = F.linear_attention_fwd(*args[:3], g, 0.7, args[3], n)
        return (o * do).sum() + (S * dS).sum()

    args = [q, k, v, S0]
    for i, grad in enumerate(grads):
        u = rng.normal(size=args[i].shape)
        diff = _difference(lambda z, i=i: loss(*args[:i], z, *args[i + 1:]), args[i], u)
        np.testing.assert_allclose((grad * u).sum(), diff, rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("shape", [(4, 9), (9, 4), (5, 5)])
def test_orthogonalize_acts_on_the_singular_values(shape):
    G = np.random.default_rng(4).normal(size=(2, *shape))
    X = F.orthogonalize(G)
    U, s, V = np.linalg.svd(G, full_matrices=False)
    s = s / (np.sqrt((s ** 2).sum(-1, keepdims=True)) + 1e-7)
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    np.testing.assert_allclose(X, U * s[:, None] @ V, atol=1e-10)
    assert s.max() < 1.3
    np.testing.assert_array_equal(F.orthogonalize(np.zeros(shape)), 0)
