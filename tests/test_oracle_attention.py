"""Pins of oracle/attention.py: closed forms, differences and invariants (no GPU)."""
import numpy as np
import pytest

from oracle import attention as A


def _difference(f, x, step=1e-6):
    g = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        for sign in (1, -1):
            y = x.copy()
            y[i] += sign * step
            g[i] += sign * f(y) / (2 * step)
    return g


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_keeps_lengths_and_depends_on_distance(layout):
    rng = np.random.default_rng(0)
    q, k, f = rng.normal(size=(5, 1, 10)), rng.normal(size=(5, 1, 10)), np.array([1.0, 0.3, 0.01])
    p = np.array([0, 1, 7, 100, 100000])
    r = A.rotate(q, p, f, layout)
    assert np.allclose((r[..., :6] ** 2).sum(-1), (q[..., :6] ** 2).sum(-1)) and np.array_equal(r[..., 6:], q[..., 6:])
    assert np.array_equal(A.rotate(q, np.zeros(5), f, layout), q)
    near = (A.rotate(q, p, f, layout) * A.rotate(k, p + 3, f, layout)).sum(-1)
    far = (A.rotate(q, p + 1000, f, layout) * A.rotate(k, p + 1003, f, layout)).sum(-1)
    assert np.allclose(near, far, atol=1e-8)
    assert np.allclose(A.rotate(r, p, f, layout, back=True), q, atol=1e-9)


def test_layouts_by_hand():
    x, p, f = np.array([[[1.0, 2.0, 3.0, 4.0]]]), np.array([1]), np.array([np.pi / 2, np.pi])
    assert np.allclose(A.rotate(x, p, f, "half"), [[[-3.0, -2.0, 1.0, -4.0]]])
    assert np.allclose(A.rotate(x, p, f, "interleaved"), [[[-2.0, 1.0, -3.0, -4.0]]])
    y = A.norm_rotary_fwd(np.full((1, 1, 4), -3.0), eps=0.0, weight=np.arange(4.0))
    assert np.allclose(y, [[[0, -1, -2, -3]]])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [True, False])
def test_rotary_gradient_by_differences(layout, norm):
    rng = np.random.default_rng(1)
    x, dy = rng.normal(size=(2, 2, 6)), rng.normal(size=(2, 2, 6))
    w = rng.normal(size=6) if norm else None
    at = dict(positions=np.array([3, 11]), frequencies=np.array([0.7, 0.1]), layout=layout, amplitude=1.2, norm=norm)
    dx, dw = A.norm_rotary_bwd(dy, x, weight=w, **at)
    assert np.allclose(dx, _difference(lambda y: (dy * A.norm_rotary_fwd(y, weight=w, **at)).sum(), x), atol=1e-7)
    if norm:
        assert np.allclose(dw, _difference(lambda y: (dy * A.norm_rotary_fwd(x, weight=y, **at)).sum(), w), atol=1e-7)


def test_attention_by_hand():
    q = np.zeros((3, 2, 2))
    k, v = np.ones((3, 1, 2)), np.arange(6.0).reshape(3, 1, 2)
    o, lse = A.packed_fwd(q, k, v, [0, 2, 3], 1.0)
    assert np.allclose(o[:, 0], [[0, 1], [1, 2], [4, 5]]) and np.allclose(o[:, 0], o[:, 1])
    assert np.allclose(lse, np.log([[1, 2, 1]] * 2))


def test_attention_gradient_by_differences():
    rng = np.random.default_rng(2)
    q, do = rng.normal(size=(2, 6, 4, 3))
    k, v = rng.normal(size=(2, 6, 2, 3))
    starts = [0, 4, 4, 6]
    for t, g in zip((0, 1, 2), A.packed_bwd(q, k, v, do, starts, 0.7)):
        def f(x):
            args = [q, k, v]
            args[t] = x
            return (do * A.packed_fwd(*args, starts, 0.7)[0]).sum()
        assert np.allclose(g, _difference(f, [q, k, v][t]), atol=1e-7)


def test_pages_give_what_the_whole_gives():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(9, 4, 5)), rng.normal(size=(9, 2, 5)), rng.normal(size=(9, 2, 5))
    want, lse = A.packed_fwd(q, k, v, [0, 9], 0.5)
    pages, table = np.full((2, 7, 4, 2, 5), np.nan), np.array([[5, 0, 3]])
    for p in range(9):
        pages[0, table[0, p // 4], p % 4], pages[1, table[0, p // 4], p % 4] = k[p], v[p]
    o, z = A.paged_fwd(q[6:], pages[0], pages[1], table, [9], [0, 3], 0.5)
    assert np.allclose(o, want[6:]) and np.allclose(z, lse[:, 6:])
    o, z = A.paged_fwd(q[:3], pages[0], pages[1], table, [1], [0, 3], 0.5)  # more rows than tokens
    assert not o[:2].any() and np.isneginf(z[:, :2]).all() and np.allclose(o[2], np.repeat(v[0], 2, axis=0))


def test_plan():
    got = A.paged_plan([0, 5, 8], [3, 4, 0], [[-1] * 3, [7, 2, -1], [1, 4, -1]], [9, 6, 3], 4, 9)
    assert got["tables"].tolist() == [[9, -1, -1], [7, 2, 6], [1, 4, -1]] and got["taken"] == [2]
    assert got["starts"].tolist() == [0, 3, 7, 7] and got["lengths"].tolist() == [3, 9, 8]
    assert got["positions"].tolist() == [0, 1, 2, 5, 6, 7, 8, 0, 0]
    assert got["slots"].tolist() == [36, 37, 38, 9, 10, 11, 24, -1, -1]
