"""Softmax attention and what stands around it in float64, from the definitions: norms of queries
and keys with the rotation by position, causal attention over packed sequences and over a paged
cache with its gradients, a paged cache's bookkeeping. With ``sizes`` the attention also returns
the same sums over absolute values, which a rounding's effect is measured by.

Test infrastructure: only tests/ use this module; the library never does.
"""
from __future__ import annotations

import numpy as np


def _pairs(R, layout):
    i = np.arange(R // 2)
    return (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)


def rotate(x, positions, frequencies, layout, amplitude=1.0, back=False):
    """Pairs of the first 2 F features of x [T,h,D] turned by positions [T] times frequencies [F]."""
    y = np.array(x, np.float64)
    if frequencies is None or len(frequencies) == 0:
        return y
    a, b = _pairs(2 * len(frequencies), layout)
    angle = np.asarray(positions, np.float64)[:, None] * np.asarray(frequencies, np.float64)
    c, s = amplitude * np.cos(angle)[:, None], amplitude * np.sin(angle)[:, None] * (-1 if back else 1)
    u, v = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return y


def norm_rotary_fwd(x, positions=None, frequencies=None, weight=None, eps=1e-6, layout="half", amplitude=1.0, norm=True):
    x = np.asarray(x, np.float64)
    if norm:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * (1 if weight is None else weight)
    return rotate(x, positions, frequencies, layout, amplitude)


def norm_rotary_bwd(dy, x, positions=None, frequencies=None, weight=None, eps=1e-6, layout="half", amplitude=1.0, norm=True):
    """(dx, dweight)."""
    g, x = rotate(dy, positions, frequencies, layout, amplitude, back=True), np.asarray(x, np.float64)
    if not norm:
        return g, None
    rstd = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    z = x * rstd
    h = g if weight is None else g * weight
    return rstd * (h - z * (h * z).mean(-1, keepdims=True)), (g * z).sum((0, 1))


def _scores(q, k, scale, before):
    """[H,n,m] scores of rows at positions before + i over keys k [m,Hk,D], -inf where a row does not see."""
    n, H, _ = q.shape
    k = np.repeat(k, H // k.shape[1], axis=1)
    s = scale * np.einsum("ihd,jhd->hij", q, k)
    s[:, np.arange(k.shape[0])[None] > before + np.arange(n)[:, None]] = -np.inf
    return s


def attend(q, k, v, scale, before=0, sizes=False):
    """Rows q [n,H,D] over keys k, v [m,Hk,D]: (o [n,H,D], lse [H,n]), with ``sizes`` also (sum p |v|, the
    rows' largest sum |q||k| scale)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    n, H, D = q.shape
    g = H // k.shape[1]
    if k.shape[0] == 0:
        o, lse = np.zeros(q.shape), np.full((H, n), -np.inf)
        return (o, lse, o, np.zeros((H, n))) if sizes else (o, lse)
    s = _scores(q, k, scale, before)
    top = s.max(-1, keepdims=True)
    p = np.exp(s - np.where(np.isfinite(top), top, 0))
    z = p.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (np.where(np.isfinite(top), top, 0) + np.log(z))[..., 0]
    p = np.divide(p, z, out=np.zeros_like(p), where=z > 0)
    vr = np.repeat(v, g, axis=1)
    o = np.einsum("hij,jhd->ihd", p, vr)
    if not sizes:
        return o, lse
    reach = abs(scale) * np.einsum("ihd,jhd->hij", np.abs(q), np.abs(np.repeat(k, g, axis=1)))
    return o, lse, np.einsum("hij,jhd->ihd", p, np.abs(vr)), np.where(np.isfinite(s), reach, 0).max(-1)


def packed_fwd(q, k, v, starts, scale, sizes=False):
    out = [np.zeros(q.shape), np.full((q.shape[1], q.shape[0]), np.nan), np.zeros(q.shape), np.zeros((q.shape[1], q.shape[0]))]
    for a, b in zip(starts[:-1], starts[1:]):
        got = attend(q[a:b], k[a:b], v[a:b], scale, 0, True)
        for t, x, heads_first in zip(out, got, (0, 1, 0, 1)):
            t[(slice(None), slice(a, b)) if heads_first else slice(a, b)] = x
    return tuple(out) if sizes else tuple(out[:2])


def packed_bwd(q, k, v, do, starts, scale, sizes=False):
    """(dq, dk, dv); with ``sizes`` also two measures of each: what a relative rounding of p and of ds moves
    (with the error of o that delta carries), and the sums over absolute values."""
    q, k, v, do = (np.asarray(t, np.float64) for t in (q, k, v, do))
    H, Hk = q.shape[1], k.shape[1]
    g = H // Hk
    out = [[np.zeros(t.shape) for t in (q, k, v)] for _ in range(3)]
    fold = lambda t: t.reshape(t.shape[0], Hk, g, -1).sum(2)  # noqa: E731
    for a, b in zip(starts[:-1], starts[1:]):
        if a == b:
            continue
        Q, K, V, G = q[a:b], np.repeat(k[a:b], g, axis=1), np.repeat(v[a:b], g, axis=1), do[a:b]
        o, lse, osize, _ = attend(q[a:b], k[a:b], v[a:b], scale, 0, True)
        p = np.exp(_scores(Q, k[a:b], scale, 0) - lse[..., None])
        dp, delta = np.einsum("ihd,jhd->hij", G, V), np.einsum("ihd,ihd->hi", G, o)
        ds = p * (dp - delta[..., None])
        # the error of o (its probabilities', and its own rounding) in delta, and magnitudes
        doff = np.einsum("ihd,ihd->hi", np.abs(G), osize + np.abs(o))
        dabs = p * (np.einsum("ihd,jhd->hij", np.abs(G), np.abs(V)) + doff[..., None])
        for kind, (w, x, mag) in enumerate(((ds, p, False), (np.abs(ds) + p * doff[..., None], p, True), (dabs, p, True))):
            f = np.abs if mag else (lambda t: t)
            out[kind][0][a:b] = abs(scale) * np.einsum("hij,jhd->ihd", w, f(K)) if mag else scale * np.einsum("hij,jhd->ihd", w, K)
            out[kind][1][a:b] = (abs(scale) if mag else scale) * fold(np.einsum("hij,ihd->jhd", w, f(Q)))
            out[kind][2][a:b] = fold(np.einsum("hij,ihd->jhd", x, f(G)))
    return out if sizes else out[0]


def gather(pages, table, n):
    """The first n tokens [n,Hk,D] of a sequence whose pages ``table`` names."""
    size = pages.shape[1]
    pos = np.arange(n)
    return pages[np.asarray(table)[pos // size], pos % size]


def paged_fwd(q, k_pages, v_pages, tables, lengths, starts, scale, sizes=False):
    out = [np.zeros(q.shape), np.full((q.shape[1], q.shape[0]), np.nan), np.zeros(q.shape), np.zeros((q.shape[1], q.shape[0]))]
    for i, (a, b) in enumerate(zip(starts[:-1], starts[1:])):
        n = int(lengths[i])
        got = attend(q[a:b], gather(k_pages, tables[i], n), gather(v_pages, tables[i], n), scale, n - (b - a), True)
        for t, x, heads_first in zip(out, got, (0, 1, 0, 1)):
            t[(slice(None), slice(a, b)) if heads_first else slice(a, b)] = x
    return tuple(out) if sizes else tuple(out[:2])


def paged_plan(cached, added, tables, free, page, tokens):
    """Request by request, token by token: dict with tables, starts, lengths, positions, slots, taken."""
    tables, W = np.array(tables), np.asarray(tables).shape[1]
    starts, positions, slots, taken = [0], [], [], 0
    for b, (n, m) in enumerate(zip(np.maximum(cached, 0), np.maximum(added, 0))):
        have, want = -(-int(n) // page), -(-int(n + m) // page)
        for col in range(have, want):
            if col < W:
                tables[b, col] = free[taken] if taken < len(free) else -1
            taken += 1
        for pos in range(int(n), int(n + m)):
            col = pos // page
            at = tables[b, col] if col < W else -1
            positions.append(pos)
            slots.append(int(at) * page + pos % page if at >= 0 else -1)
        starts.append(len(slots))
    positions, slots = positions[:tokens], slots[:tokens]
    pad = tokens - len(slots)
    return dict(tables=tables, starts=np.array(starts), lengths=np.maximum(cached, 0) + np.maximum(added, 0),
                positions=np.array(positions + [0] * pad), slots=np.array(slots + [-1] * pad), taken=np.array([taken]))
