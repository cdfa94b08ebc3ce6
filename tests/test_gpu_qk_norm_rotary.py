"""GPU parity of the norms of queries and keys with the rotation by position (pc_qk_norm_rotary_fwd / _bwd)
against float64: both layouts, part of the head, odd sizes, far positions, strides, in place.

Tolerances. u = 2^-24. A norm's sum over D squares, its root and the products pass at most D / 2 + 12
roundings relative to |u_a| + |u_b|, the size of a rotated feature; the angle's cosine and sine are off by 2^-22
in float32 (the turn's fraction rounded to 24 bits: pi 2^-24; the function: 2^-23) and 2^-20 in bf16, whose output
is rounded by 2^-8 relative. A weight's gradient sums one term a row, in a tree of no more than 64 + rows / 64
additions a term, and carries each term's own roundings."""
import numpy as np
import pytest
import torch

import log_space_sum_gb300 as pc
from oracle import attention as A

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pc.load()


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _draw(T, H, Hk, D, R, dtype, seed, far=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, dq = (r(T, H, D).to(TYPES[dtype]) for _ in range(2))
    k, dk = (r(T, Hk, D).to(TYPES[dtype]) for _ in range(2))
    w = [1 + 0.3 * r(D) for _ in range(2)]
    pos = torch.randint(-5, 1 << 30 if far else 3000, (T,), generator=g, device="cuda", dtype=torch.int32)
    f = pc.rotary_frequencies(R)[0] if R else None
    return q, k, dq, dk, w, (pos if R else None), f


def _size(x, R, layout):
    """|u_a| + |u_b| of each rotated feature's pair, |u| elsewhere."""
    z = np.abs(x)
    if R:
        a, b = A._pairs(R, layout)
        both = z[..., a] + z[..., b]
        z[..., a], z[..., b] = both, both
    return z


def _tol(size, want, D, dtype):
    bf = dtype == "bf16"
    return size * ((D / 2 + 12) * U + (2.0 ** -20 if bf else 2.0 ** -22)) + (2.0 ** -8 * np.abs(want) if bf else 0) + 1e-30


def _check(q, k, dq, dk, w, pos, f, dtype, layout="half", norm=True, amplitude=1.0, eps=1e-6, out=None):
    D, R = q.shape[-1], 0 if f is None else 2 * f.shape[0]
    ws = w if norm else [None, None]
    at = dict(eps=eps, layout=layout, amplitude=amplitude, norm=norm)
    got = pc.qk_norm_rotary_fwd(q, k, pos, f, *ws, **at)
    P, F = _np(pos), _np(f)
    for x, wt, y in zip((q, k), ws, got):
        X, W = _np(x), _np(wt)
        want = A.norm_rotary_fwd(X, P, F, W, **at)
        plain = A.norm_rotary_fwd(X, weight=W, eps=eps, norm=norm)
        size = _size(plain, R, layout) * max(1, abs(amplitude))
        assert np.all(np.abs(_np(y) - want) <= _tol(size, want, D, dtype))
    back = pc.qk_norm_rotary_bwd(dq, dk, q, k, pos, f, *ws, **at, **(out or {}))
    for n, x, g, wt in (("q", q, dq, ws[0]), ("k", k, dk, ws[1])):
        X, G, W = _np(x), _np(g), _np(wt)
        dx, dw = A.norm_rotary_bwd(G, X, P, F, W, **at)
        size = _size(G, R, layout) * max(1, abs(amplitude))
        rows = G.shape[0] * G.shape[1]
        if norm:
            rstd = 1 / np.sqrt((X ** 2).mean(-1, keepdims=True) + eps)
            z = np.abs(X * rstd)
            terms = (D + 30 + 64 + rows / 64) * U + (2.0 ** -20 if dtype == "bf16" else 2.0 ** -22)
            assert np.all(np.abs(_np(back[f"d{n}_weight"]) - dw) <= terms * (size * z).sum((0, 1)) + 1e-30), n
            h = size * np.abs(W) if W is not None else size
            size = rstd * (h + z * (h * z).mean(-1, keepdims=True)) * 2  # the sums' roundings and the norm's own
        else:
            assert back[f"d{n}_weight"] is None
        assert np.all(np.abs(_np(back[f"d{n}"]) - dx) <= _tol(size, dx, D, dtype)), n
    return got, back


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,Hk,D,R", [
    (1, 1, 1, 1, 0), (1, 4, 1, 2, 2), (7, 3, 1, 64, 64), (5, 8, 2, 128, 128), (64, 5, 5, 128, 96), (3, 2, 2, 40, 20),
    (9, 6, 3, 72, 72), (33, 1, 1, 17, 6), (2, 3, 2, 255, 100), (4, 2, 1, 256, 256), (300, 2, 1, 80, 80), (6, 7, 2, 96, 32),
    (3, 4, 2, 130, 66), (2, 70, 1, 16, 8)])
def test_sizes(T, H, Hk, D, R, layout, dtype):
    x = _draw(T, H, Hk, D, R, dtype, T + D + R)
    _check(*x, dtype, layout)
    if R:
        _check(*x, dtype, layout, norm=False, amplitude=1.25)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_far_positions_and_weights_of_none(dtype):
    q, k, dq, dk, w, pos, f = _draw(40, 4, 2, 128, 128, dtype, 3, far=True)
    _check(q, k, dq, dk, w, pos, f, dtype)
    pos[0], pos[1] = 2 ** 31 - 1, -2 ** 31
    _check(q, k, dq, dk, [None, None], pos, f, dtype, "interleaved", amplitude=0.7)
    # frequencies at the ends: zero, tiny, many turns a position, negative
    f = torch.tensor([0.0, 1e-30, 1e-7, 3.0, 700.0, -0.3, -1e-3, 6.2831853], device="cuda")
    pos = torch.arange(40, device="cuda", dtype=torch.int32) * 1000
    _check(q, k, dq, dk, w, pos, f, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_strides_in_place_and_unaligned(dtype, layout):
    T, H, Hk, D = 21, 4, 2, 64
    q, k, dq, dk, w, pos, f = _draw(T, H, Hk, D, D, dtype, 4)
    want, wback = _check(q, k, dq, dk, w, pos, f, dtype, layout)
    proj = torch.empty(T, (H + 2 * Hk) * D, dtype=TYPES[dtype], device="cuda")
    cut = lambda p: (p[:, :H * D].unflatten(-1, (H, D)), p[:, H * D:(H + Hk) * D].unflatten(-1, (Hk, D)))  # noqa: E731
    qs, ks = cut(proj)
    qs.copy_(q), ks.copy_(k)
    grads = cut(torch.empty_like(proj))
    got, back = _check(qs, ks, dq, dk, w, pos, f, dtype, layout, out=dict(dq=grads[0], dk=grads[1]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(torch.equal(back[n], wback[n]) for n in wback)
    inplace = pc.qk_norm_rotary_fwd(qs, ks, pos, f, *w, layout=layout, q_out=qs, k_out=ks)
    assert inplace[0] is qs and torch.equal(qs, want[0]) and torch.equal(ks, want[1])
    g = [dq.clone(), dk.clone()]
    again = pc.qk_norm_rotary_bwd(*g, q, k, pos, f, *w, layout=layout, dq=g[0], dk=g[1])
    assert all(torch.equal(again[n], wback[n]) for n in wback)
    odd = [torch.empty(T, h, D + 1, dtype=TYPES[dtype], device="cuda")[..., 1:].copy_(t) for h, t in ((H, q), (Hk, k))]
    _check(*odd, dq, dk, w, pos, f, dtype, layout)
    heads_first = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k)]
    got, _ = _check(*heads_first, dq, dk, w, pos, f, dtype, layout)
    assert torch.equal(got[0], want[0])


def test_one_side_only_accumulate_and_repeat():
    q, k, dq, dk, w, pos, f = _draw(4097, 3, 1, 128, 64, "bf16", 5)
    _check(q, k[:, :0], dq, dk[:, :0], w, pos, f, "bf16")
    _check(q[:, :0], k, dq[:, :0], dk, w, pos, f, "bf16")
    one = pc.qk_norm_rotary_bwd(dq, dk, q, k, pos, f, *w)
    two = pc.qk_norm_rotary_bwd(dq, dk, q, k, pos, f, *w)
    assert all(torch.equal(one[n], two[n]) for n in one)
    sums = [one["dq_weight"].clone(), one["dk_weight"].clone()]
    pc.qk_norm_rotary_bwd(dq, dk, q, k, pos, f, *w, dq_weight=sums[0], dk_weight=sums[1], accumulate=True)
    assert torch.equal(sums[0], 2 * one["dq_weight"]) and torch.equal(sums[1], 2 * one["dk_weight"])


def test_rows_of_zeros_and_what_is_not_finite():
    q, k, dq, dk, w, pos, f = _draw(6, 2, 2, 64, 64, "fp32", 6)
    q[1], k[2, 0] = 0, float("nan")
    got = pc.qk_norm_rotary_fwd(q, k, pos, f, *w)
    assert not got[0][1].any() and torch.isnan(got[1][2, 0]).all()
    assert torch.isfinite(got[1][2, 1]).all() and torch.isfinite(got[1][3]).all()  # other rows do not see it
    back = pc.qk_norm_rotary_bwd(dq, dk, q, k, pos, f, *w)
    assert torch.isfinite(back["dq"]).all() and torch.isfinite(back["dk"][:2]).all()


def test_empty():
    q, k, dq, dk, w, pos, f = _draw(0, 2, 1, 64, 64, "bf16", 7)
    assert pc.qk_norm_rotary_fwd(q, k, pos, f, *w)[0].shape == (0, 2, 64)
    got = pc.qk_norm_rotary_bwd(dq, dk, q, k, pos, f, *w)
    assert got["dq"].shape == (0, 2, 64) and not got["dq_weight"].any() and not got["dk_weight"].any()


def test_refusals():
    q, k, dq, dk, w, pos, f = _draw(4, 2, 1, 64, 64, "bf16", 8)
    with pytest.raises(ValueError, match="unknown layout"):
        pc.qk_norm_rotary_fwd(q, k, pos, f, layout="both")
    with pytest.raises(ValueError, match="k has shape"):
        pc.qk_norm_rotary_fwd(q, k[:3], pos, f)
    with pytest.raises(TypeError, match="k must be torch.bfloat16"):
        pc.qk_norm_rotary_fwd(q, k.float(), pos, f)
    with pytest.raises(ValueError, match="need positions"):
        pc.qk_norm_rotary_fwd(q, k, None, f)
    with pytest.raises(TypeError, match="positions must be torch.int32"):
        pc.qk_norm_rotary_fwd(q, k, pos.long(), f)
    with pytest.raises(ValueError, match="weights need norm"):
        pc.qk_norm_rotary_fwd(q, k, pos, f, w[0], norm=False)
    with pytest.raises(ValueError, match="q_weight has shape"):
        pc.qk_norm_rotary_fwd(q, k, pos, f, w[0][:32])
    with pytest.raises(pc.PCError, match="rotated features"):
        pc.qk_norm_rotary_fwd(q, k, pos, torch.ones(33, device="cuda"))
    with pytest.raises(pc.PCError, match="other strides"):
        pc.qk_norm_rotary_fwd(q, k, pos, f, q_out=q.as_strided(q.shape, (64, 256, 1)))
    with pytest.raises(ValueError, match="accumulate needs"):
        pc.qk_norm_rotary_bwd(dq, dk, q, k, pos, f, *w, accumulate=True)
