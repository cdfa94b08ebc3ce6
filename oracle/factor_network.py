"""The factor network's operators in float64: layer norm, linear attention with a decay for
each head, orthogonalised updates, and their gradients, from their definitions.

Test infrastructure: only tests/ use this module; the library never does.
"""
from __future__ import annotations

import numpy as np


def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5):
    """Rows of x normalised: (y, mean, rstd)."""
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    rstd = 1 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layer_norm_bwd(dy, x, weight, mean, rstd):
    """(dx, dweight, dbias) from the forward's statistics."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    z = (x - mean[..., None]) * rstd[..., None]
    g = dy if weight is None else dy * weight
    dx = rstd[..., None] * (g - g.mean(-1, keepdims=True) - z * (g * z).mean(-1, keepdims=True))
    rows = tuple(range(x.ndim - 1))
    return dx, (dy * z).sum(rows), dy.sum(rows)


def _decay(log_decay):
    return np.exp(np.asarray(log_decay, np.float64))[None, :, None, None]


def _there(lengths, B, T):
    n = np.full(B, T) if lengths is None else np.clip(lengths, 0, T)
    return np.arange(T) < n[:, None]


def linear_attention_fwd(q, k, v, log_decay, scale=1.0, state=None, lengths=None):
    """S_t = l S_{t-1} + k_t v_t^T, o_t = scale q_t^T S_t, one token after the other: q, k
    [B,T,H,Dk], v [B,T,H,Dv]. Returns (o, S after each sequence's last token)."""
    B, T, H, dk = q.shape
    S = np.zeros((B, H, dk, v.shape[-1])) if state is None else np.array(state, np.float64)
    lam, there = _decay(log_decay), _there(lengths, B, T)
    o = np.zeros((B, T, H, v.shape[-1]))
    for t in range(T):
        on = there[:, t]
        S[on] = lam * S[on] + k[on, t, :, :, None] * v[on, t, :, None, :]
        o[on, t] = scale * np.einsum("bhk,bhkv->bhv", q[on, t], S[on])
    return o, S


def linear_attention_bwd(q, k, v, log_decay, do, scale=1.0, state=None, dstate=None, lengths=None):
    """(dq, dk, dv, gradient of the initial state), by reversing the recurrence."""
    B, T, H, dk = q.shape
    lam, there = _decay(log_decay), _there(lengths, B, T)
    S = np.zeros((B, H, dk, v.shape[-1])) if state is None else np.array(state, np.float64)
    dq, dkk, dvv = (np.zeros(x.shape) for x in (q, k, v))
    for t in range(T):
        on = there[:, t]
        S[on] = lam * S[on] + k[on, t, :, :, None] * v[on, t, :, None, :]
        dq[on, t] = scale * np.einsum("bhkv,bhv->bhk", S[on], do[on, t])
    R = np.zeros_like(S) if dstate is None else np.array(dstate, np.float64)
    for t in reversed(range(T)):
        on = there[:, t]
        R[on] += scale * q[on, t, :, :, None] * do[on, t, :, None, :]
        dkk[on, t] = np.einsum("bhkv,bhv->bhk", R[on], v[on, t])
        dvv[on, t] = np.einsum("bhkv,bhk->bhv", R[on], k[on, t])
        R[on] = lam * R[on]
    return dq, dkk, dvv, R


def orthogonalize(G, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7):
    """Newton-Schulz products on G / (|G|_F + eps), matrices in the last two dimensions."""
    X = np.asarray(G, np.float64)
    X = X / (np.sqrt((X ** 2).sum((-1, -2), keepdims=True)) + eps)
    tall = X.shape[-2] > X.shape[-1]
    X = X.swapaxes(-1, -2) if tall else X
    a, b, c = coefficients
    for _ in range(steps):
        A = X @ X.swapaxes(-1, -2)
        X = a * X + (b * A + c * A @ A) @ X
    return X.swapaxes(-1, -2) if tall else X
