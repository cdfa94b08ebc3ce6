"""GPU parity of layer norm (pc_layer_norm_fwd / _bwd) against the float64 oracle: row
lengths around every variant's limits, odd and unaligned rows, strides, one row, offsets
far larger than the spread, non-finite rows.

Tolerances. u = 2^-24. A float32 row sum of a thread's few values and a tree over them adds
at most about 32 roundings, so the centred values carry 32 u max|x|, and a value of y
(32 u max|x| + 8 u |x - mean|) rstd |w| + 4 u |y|; the sums over rows of the weight's gradient add
one rounding for each row that a CTA takes. bf16 outputs add half a unit in the last
place, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import log_space_sum_gb300 as pc
from oracle import factor_network as F

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
HALF_ULP = {"fp32": 2 * U, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pc.load()


def _np(t):
    return t.detach().double().cpu().numpy()


def _draw(rows, dim, dtype, seed, offset=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return (r(rows, dim) + offset).to(TYPES[dtype]), r(rows, dim).to(TYPES[dtype]), 1 + 0.3 * r(dim), 0.3 * r(dim)


def _check_fwd(x, w, b, got, dtype, eps=1e-5):
    y, mean, rstd = (_np(t) for t in got)
    X, W, Bi = _np(x), None if w is None else _np(w), None if b is None else _np(b)
    ry, rm, rr = F.layer_norm_fwd(X, W, Bi, eps)
    top = np.abs(X).max(-1, keepdims=True)
    tol = (32 * U * top + 8 * U * np.abs(X - rm[..., None])) * rr[..., None] * (1 if W is None else np.abs(W)) \
        + (4 * U + HALF_ULP[dtype]) * np.abs(ry) + (0 if Bi is None else 2 * U * np.abs(Bi))
    assert np.all(np.abs(y - ry) <= tol)
    assert np.all(np.abs(mean - rm) <= 32 * U * top[..., 0])
    # d rstd / rstd = -(err of the centred values) . z / D, at most err * rstd
    assert np.all(np.abs(rstd - rr) <= rr * (40 * U + 64 * U * top[..., 0] * rr))


def _check_bwd(x, dy, w, mean, rstd, got, dtype):
    dx, dw, db = (_np(t) for t in got)
    X, G, M, R = _np(x), _np(dy), _np(mean), _np(rstd)
    W = None if w is None else _np(w)
    rx, rw, rb = F.layer_norm_bwd(G, X, W, M, R)
    z = np.abs((X - M[..., None]) * R[..., None])
    ez = 2 * U * np.abs(X) * R[..., None] + 2 * U * z
    g = np.abs(G if W is None else G * W)
    avg = lambda t: t.mean(-1, keepdims=True)  # noqa: E731
    tol = R[..., None] * (4 * U * g + 40 * U * avg(g) + 44 * U * z * avg(g * z) + ez * avg(g * z) + z * avg(g * ez)) \
        + (4 * U + HALF_ULP[dtype]) * np.abs(rx)
    assert np.all(np.abs(dx - rx) <= tol)
    n = X.reshape(-1, X.shape[-1]).shape[0]
    chain = min(n, -(-n // 152) + 600)
    flat = lambda t: np.abs(t).reshape(-1, X.shape[-1]).sum(0)  # noqa: E731
    assert np.all(np.abs(dw - rw) <= chain * U * flat(G * z) + flat(G * ez))
    assert np.all(np.abs(db - rb) <= chain * U * flat(G))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (5, 8), (2, 64), (33, 256), (7, 260), (130, 512), (9, 768),
                                      (4, 1024), (5, 1537), (3, 2048), (700, 1032), (3, 4096), (2, 8192),
                                      (2, 8200), (2, 16384), (2, 20001)])
def test_sizes(rows, dim, dtype):
    x, dy, w, b = _draw(rows, dim, dtype, rows * 131 + dim)
    got = pc.layer_norm_fwd(x, w, b)
    _check_fwd(x, w, b, got, dtype)
    _check_bwd(x, dy, w, got[1], got[2], pc.layer_norm_bwd(dy, x, w, got[1], got[2]), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_without_parameters_and_leading_dimensions(dtype):
    x, dy, w, b = _draw(12, 96, dtype, 5)
    x, dy = x.view(3, 4, 96), dy.view(3, 4, 96)
    got = pc.layer_norm_fwd(x)
    assert got[0].shape == x.shape and got[1].shape == x.shape[:-1]
    _check_fwd(x, None, None, got, dtype)
    dx, dw, db = pc.layer_norm_bwd(dy, x, None, got[1], got[2])
    _check_bwd(x, dy, None, got[1], got[2], (dx, dw, db), dtype)
    only = pc.layer_norm_bwd(dy, x, None, got[1], got[2], params=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], dx)
    dw2, db2 = torch.ones_like(dw), torch.ones_like(db)
    pc.layer_norm_bwd(dy, x, None, got[1], got[2], dweight=dw2, dbias=db2, accumulate=True)
    assert torch.equal(dw2, dw + 1) and torch.equal(db2, db + 1)
    w4 = pc.layer_norm_fwd(x, w)  # a weight and no bias
    _check_fwd(x, w, None, w4, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
def test_strided_rows(dtype, shift):
    """Rows cut from a wider matrix, from an aligned and from an unaligned column."""
    wide, gwide, w, b = _draw(37, 640, dtype, 6)
    x, dy = wide[:, shift:shift + 256], gwide[:, shift:shift + 256]
    out = torch.zeros_like(wide)
    got = pc.layer_norm_fwd(x, w[:256], b[:256], out=out[:, shift:shift + 256])
    _check_fwd(x, w[:256], b[:256], got, dtype)
    dwide = torch.zeros_like(wide)
    _check_bwd(x, dy, w[:256], got[1], got[2],
               pc.layer_norm_bwd(dy, x, w[:256], got[1], got[2], dx=dwide[:, shift:shift + 256]), dtype)
    for t in (out, dwide):  # nothing beside the rows was written
        assert not t[:, shift + 256:].any() and not t[:, :shift].any()
    # a parameter that does not start on 16 bytes
    _check_fwd(x, w[1:257], b[1:257], pc.layer_norm_fwd(x, w[1:257], b[1:257]), dtype)


def test_large_offset_constant_rows_and_empty():
    x, _, w, b = _draw(6, 512, "fp32", 7, offset=1e4)
    _check_fwd(x, w, b, pc.layer_norm_fwd(x, w, b), "fp32")
    flat = torch.full((2, 512), 3.0, device="cuda")
    y, mean, rstd = pc.layer_norm_fwd(flat, w, b)
    assert torch.equal(y, b.expand(2, -1)) and torch.equal(mean, flat[:, 0])
    np.testing.assert_allclose(_np(rstd), 1e-5 ** -0.5, rtol=1e-6)
    none = torch.empty(0, 512, device="cuda")
    y, mean, rstd = pc.layer_norm_fwd(none, w, b)
    assert y.shape == none.shape
    _, dw, db = pc.layer_norm_bwd(none, none, w, mean, rstd)
    assert not dw.any() and not db.any()


def test_a_non_finite_row_stays_alone():
    x, _, w, b = _draw(9, 1024, "bf16", 8)
    x[4, 17] = float("nan")
    x[6, 3] = float("inf")
    y = pc.layer_norm_fwd(x, w, b)[0]
    bad = torch.isnan(y).all(-1)
    assert bad.tolist() == [i in (4, 6) for i in range(9)]
    assert torch.isfinite(y[~bad]).all()


def test_in_place_repeats_and_streams():
    x, dy, w, b = _draw(300, 1024, "bf16", 9)
    want = pc.layer_norm_fwd(x, w, b)
    grads = pc.layer_norm_bwd(dy, x, w, want[1], want[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = pc.layer_norm_bwd(dy, x, w, want[1], want[2])
        x2, dy2 = x.clone(), dy.clone()
        pc.layer_norm_bwd(dy2, x2, w, want[1], want[2], dx=dy2)
        pc.layer_norm_fwd(x2, w, b, out=x2)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(grads, again))
    assert torch.equal(x2, want[0]) and torch.equal(dy2, grads[0])


def test_refusals():
    x, dy, w, b = _draw(4, 64, "bf16", 10)
    mean = torch.empty(4, device="cuda")
    with pytest.raises(TypeError, match="x must be torch.float32 or"):
        pc.layer_norm_fwd(x.half(), w, b)
    with pytest.raises(ValueError, match="weight has shape"):
        pc.layer_norm_fwd(x, w[:63], b)
    with pytest.raises(TypeError, match="bias must be torch.float32"):
        pc.layer_norm_fwd(x, w, b.bfloat16())
    with pytest.raises(ValueError, match="contiguous along its last"):
        pc.layer_norm_fwd(x.t(), w[:4], b[:4])
    with pytest.raises(TypeError, match="dy must be torch.bfloat16"):
        pc.layer_norm_bwd(dy.float(), x, w, mean, mean)
    with pytest.raises(ValueError, match="accumulate needs"):
        pc.layer_norm_bwd(dy, x, w, mean, mean, accumulate=True)
    with pytest.raises(pc.PCError, match="eps"):
        pc.layer_norm_fwd(x, w, b, eps=-1.0)
    with pytest.raises(ValueError, match="collapse"):
        pc.layer_norm_fwd(torch.empty(4, 6, 64, device="cuda")[:, :3], w, b)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,dim,ld,first", [(1, 3, 11, 5), (9, 13, 13, 0), (17, 65, 77, 3), (40, 511, 640, 1), (300, 257, 263, 6),
                                               (2500, 1031, 1033, 7), (1300, 1537, 1537, 0), (50, 4091, 4097, 2),
                                               (20, 8190, 8191, 4), (9000, 100, 101, 1)])
def test_rows_that_start_and_end_inside_a_piece(rows, dim, ld, first, dtype):
    """Rows ld values apart from an odd place: the values around them are NaN in the inputs and
    stay as they are in the outputs. Outputs placed as the inputs, and one value further."""
    x, dy, w, b = _draw(rows, dim, dtype, rows + dim)

    def inside(t, shift=0, fill=float("nan")):
        flat = torch.full((first + shift + rows * ld + 16,), fill, dtype=t.dtype, device="cuda")
        view = flat[first + shift:first + shift + rows * ld].view(rows, ld)[:, :dim]
        if t is not None:
            view.copy_(t)
        return flat, view

    xv, dv = inside(x)[1], inside(dy)[1]
    results = []
    for shift in (0, 1):
        flat, out = inside(torch.zeros_like(x), shift, 7.0)
        got = pc.layer_norm_fwd(xv, w, b, out=out)
        _check_fwd(x, w, b, got, dtype)
        flat2, dx = inside(torch.zeros_like(x), shift, 7.0)
        grads = pc.layer_norm_bwd(dv, xv, w, got[1], got[2], dx=dx)
        _check_bwd(x, dy, w, got[1], got[2], grads, dtype)
        for f, view in ((flat, out), (flat2, dx)):
            view.fill_(7.0)
            assert (f == 7.0).all()
        results.append(got[1:])
    again = pc.layer_norm_bwd(dv, xv, w, *results[0])
    more = pc.layer_norm_bwd(dv, xv, w, *results[0])
    assert all(torch.equal(p, q) for p, q in zip(again, more))
