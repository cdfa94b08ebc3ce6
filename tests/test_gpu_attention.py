"""GPU parity of causal softmax attention over packed sequences (pc_attention_fwd / _bwd) against float64: head
sizes on both sides of the tensor-core kernels' limits, groups of heads, lengths of zero, one and past several
tiles, strides, what lies between and behind sequences.

Tolerances. u = 2^-24. A score's sum over D products, scaled, is off by (D + 8) u times the sum of their
magnitudes (E: its largest in a row, scaled), and moves p by twice that, relative; sums over the keys pass n + 16
more roundings. With bf16 elements p is rounded once (2^-8 of each term) and the output once more; as these
roundings are independent, the 2-norm of o's error is three times 1.7e-3 (a bf16 rounding's root mean
square) at most. In the gradients p and ds are rounded once each, and delta carries the forward's output, with its
own roundings; the oracle measures all three."""
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
    yield
    pc.device_status()


def _np(t):
    return t.detach().double().cpu().numpy()


def _draw(T, H, Hk, D, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda h: torch.randn(T, h, D, generator=g, device="cuda").to(TYPES[dtype])  # noqa: E731
    return r(H), r(Hk), r(Hk), r(H)


def _starts(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)


def _int(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _close(got, want, tol, what, rms=None):
    got = _np(got) if isinstance(got, torch.Tensor) else got
    assert np.isfinite(got).all(), what
    assert np.all(np.abs(got - want) <= tol + 1e-30), what
    if rms is not None:
        assert np.linalg.norm(got - want) <= rms * np.linalg.norm(want) + 1e-30, what


def check(q, k, v, do, lengths, dtype, scale=None, packed=True, **out):
    """Both directions against the oracle; returns (o, lse, gradients)."""
    bf, D = dtype == "bf16", q.shape[-1]
    s = D ** -0.5 if scale is None else scale
    starts = _starts(lengths)
    dev = _int(starts) if packed else None
    Q, K, V, G = (_np(t) for t in (q, k, v, do))
    o, lse = pc.attention_fwd(q, k, v, starts=dev, scale=scale)
    n = int(starts[-1])
    ro, rl, size, reach = A.packed_fwd(Q, K, V, starts, s, sizes=True)
    E = (D + 8) * U * reach
    longest = max(list(lengths) + [1])
    move = 2 * E.T[..., None] + (longest + 16) * U
    _close(_np(o)[:n], ro[:n], (size * move + (2.0 ** -8 * (size + np.abs(ro)) if bf else 0))[:n], "o",
           3 * 1.7e-3 if bf else None)
    _close(_np(lse)[:, :n], rl[:, :n], (E + (longest + 16 + 2 * np.abs(rl)) * U)[:, :n], "lse")
    got = pc.attention_bwd(q, k, v, o, lse, do, starts=dev, scale=scale, **out)
    want, rounded, mag = A.packed_bwd(Q, K, V, G, starts, s, sizes=True)
    top = 2 * E.max(initial=0) + (longest * (q.shape[1] // k.shape[1]) + D + 24 + 2 * np.abs(rl[:, :n]).max(initial=0)) * U
    for name, w, r, m in zip(("dq", "dk", "dv"), want, rounded, mag):
        tol = 2 * m * top + (2.0 ** -8 * (r + np.abs(w)) if bf else 0)
        _close(_np(got[name])[:n], w[:n], tol[:n], name)
    return o, lse, got


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,H,Hk,D", [
    (1, 1, 1, 1), (1, 8, 1, 128), (2, 3, 3, 64), (5, 4, 2, 3), (33, 2, 1, 40), (64, 6, 2, 64), (127, 2, 2, 128),
    (128, 8, 4, 64), (129, 4, 1, 128), (257, 5, 1, 72), (300, 3, 1, 96), (130, 7, 1, 8), (90, 4, 2, 200), (70, 2, 1, 256),
    (513, 16, 2, 128), (640, 2, 1, 64), (65, 33, 1, 16), (50, 17, 1, 128), (385, 12, 1, 120), (260, 2, 2, 36)])
def test_one_sequence(T, H, Hk, D, dtype):
    check(*_draw(T, H, Hk, D, dtype, T + H + D), [T], dtype, packed=bool(T % 2))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lengths", [[300, 0, 1, 129], [0, 0, 0], [1] * 70, [128, 127, 2, 256], [7, 600, 0, 33, 64, 0]])
@pytest.mark.parametrize("H,Hk,D", [(4, 2, 64), (3, 1, 128), (2, 2, 80)])
def test_packed_lengths(lengths, H, Hk, D, dtype):
    check(*_draw(sum(lengths), H, Hk, D, dtype, 11), lengths, dtype, scale=0.2)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B", [128, 129, 300])
@pytest.mark.parametrize("H,Hk,D", [(4, 1, 128), (2, 2, 40)])
def test_many_sequences(B, H, Hk, D, dtype):
    rng = np.random.default_rng(B)
    lengths = rng.integers(0, 9, B) * (rng.random(B) < 0.8)
    lengths[[5, B // 2, B - 1]] = 200, 131, 257
    check(*_draw(int(lengths.sum()), H, Hk, D, dtype, B), lengths.tolist(), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 36])
def test_sequences_do_not_see_one_another_nor_what_lies_behind(dtype, D):
    lengths, T = [130, 61, 257], 500
    q, k, v, do = _draw(T, 4, 2, D, dtype, 12)
    o, lse, got = check(q, k, v, do, lengths, dtype)
    n, a, b = sum(lengths), 130, 191
    for t in (q, k, v, do):  # the sequence in the middle, and the rows behind the last
        t[a:b] = float("nan")
        t[n:] = float("inf")
    starts = _int(_starts(lengths))
    o2, l2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    pc.attention_fwd(q, k, v, starts=starts, out=o2, lse=l2)
    grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
    back = pc.attention_bwd(q, k, v, o2, l2, do, starts=starts, dq=grads[0], dk=grads[1], dv=grads[2])
    for part in (slice(0, a), slice(b, n)):
        assert torch.equal(o2[part], o[part]) and torch.equal(l2[:, part], lse[:, part])
        assert all(torch.equal(back[x][part], got[x][part]) for x in got)
    for t in (o2, *grads):
        assert (t[n:] == 7.0).all()
    assert (l2[:, n:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("layout", ["projection", "heads first", "unaligned", "shared"])
def test_strides(dtype, layout):
    T, H, Hk, D, lengths = 290, 4, 2, 64, [150, 140]
    q, k, v, do = _draw(T, H, Hk, D, dtype, 13)
    want = check(q, k, v, do, lengths, dtype)
    dt, out = TYPES[dtype], {}
    if layout == "projection":
        cut = lambda p: (p[:, :H * D].unflatten(-1, (H, D)), p[:, H * D:(H + Hk) * D].unflatten(-1, (Hk, D)),  # noqa: E731
                         p[:, (H + Hk) * D:].unflatten(-1, (Hk, D)))
        parts = cut(torch.empty(T, (H + 2 * Hk) * D, device="cuda", dtype=dt))
        out = dict(zip(("dq", "dk", "dv"), cut(torch.empty(T, (H + 2 * Hk) * D, device="cuda", dtype=dt))))
    elif layout == "heads first":
        parts = [torch.empty(h, T, D, device="cuda", dtype=dt).transpose(0, 1) for h in (H, Hk, Hk)]
    elif layout == "unaligned":
        parts = [torch.empty(T, h, D + 1, device="cuda", dtype=dt)[..., 1:] for h in (H, Hk, Hk)]
    else:  # one head of keys and values for all, without a copy: each head's gradient is its own
        check(q, k[:, :1].expand(-1, Hk, -1), v[:, :1].expand(-1, Hk, -1), do, lengths, dtype)
        check(q[:, :1].expand(-1, H, -1), k, v, do[:1].expand(T, -1, -1), lengths, dtype)
        return
    for p, t in zip(parts, (q, k, v)):
        p.copy_(t)
    got = check(*parts, do, lengths, dtype, **out)
    if layout != "unaligned":
        assert torch.equal(got[0], want[0]) and all(torch.equal(got[2][n], want[2][n]) for n in want[2])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_that_span_the_range(dtype, D):
    """Running maxima that rise late, scores of hundreds, and a scale of zero and below it."""
    T = 400
    q, k, v, do = _draw(T, 2, 1, D, dtype, 14)
    k *= torch.linspace(0.1, 12, T, device="cuda").to(k.dtype)[:, None, None]
    check(q, k, v, do, [T], dtype, scale=1.0)
    check(q, k, v, do, [T], dtype, scale=-0.5)
    o, lse, _ = check(q, k, v, do, [T], dtype, scale=0.0)
    assert torch.allclose(lse[0].exp(), torch.arange(1, T + 1, device="cuda").float(), rtol=1e-5)
    k.neg_()  # ... and that fall
    check(q, k, v, do, [T], dtype, scale=1.0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_what_is_not_finite_stays_with_the_rows_that_see_it(dtype):
    T, at = 700, 300
    q, k, v, do = _draw(T, 2, 1, 128, dtype, 15)
    want, _ = pc.attention_fwd(q, k, v)
    k[at] = float("nan")
    o, lse = pc.attention_fwd(q, k, v)
    assert torch.equal(o[:at], want[:at]) and torch.isnan(o[at:]).all() and torch.isnan(lse[:, at:]).all()
    k[at], q[at + 5] = 0, float("nan")
    o, _ = pc.attention_fwd(q, k, v)
    assert torch.isnan(o[at + 5]).all() and torch.isfinite(o[:at + 5]).all() and torch.isfinite(o[at + 6:]).all()
    q[at + 5], v[at] = 0, float("inf")
    o, _ = pc.attention_fwd(q, k, v)
    assert torch.isfinite(o[:at - 127]).all() and not torch.isfinite(o[at:]).any()


def test_a_layer_of_them_by_differences():
    """Norms with rotation, attention and back, float32: the gradients' products with a direction are the loss's
    differences along it (in float64; the kernels' own error is 1e-5 of the sums' magnitudes)."""
    T, H, Hk, D, starts = 150, 4, 2, 40, [0, 90, 150]
    q, k, v, do = _draw(T, H, Hk, D, "fp32", 20)
    w = [1 + 0.2 * torch.randn(D, device="cuda") for _ in range(2)]
    pos, (f, _), dev = torch.arange(T, device="cuda", dtype=torch.int32) * 3, pc.rotary_frequencies(24), _int(starts)
    qr, kr = pc.qk_norm_rotary_fwd(q, k, pos, f, *w)
    o, lse = pc.attention_fwd(qr, kr, v, starts=dev)
    back = pc.attention_bwd(qr, kr, v, o, lse, do, starts=dev)
    first = pc.qk_norm_rotary_bwd(back["dq"], back["dk"], q, k, pos, f, *w)
    got = [first["dq"], first["dk"], back["dv"], first["dq_weight"], first["dk_weight"]]
    P, F, G = _np(pos), _np(f), _np(do)

    def loss(q, k, v, wq, wk):
        qr, kr = A.norm_rotary_fwd(q, P, F, wq), A.norm_rotary_fwd(k, P, F, wk)
        return (G * A.packed_fwd(qr, kr, v, starts, D ** -0.5)[0]).sum()

    at, rng = [_np(t) for t in (q, k, v, *w)], np.random.default_rng(1)
    for i, g in enumerate(got):
        d, step = rng.normal(size=at[i].shape), 1e-5
        plus, minus = ([x + sign * step * d if j == i else x for j, x in enumerate(at)] for sign in (1, -1))
        want = (loss(*plus) - loss(*minus)) / (2 * step)
        assert abs((_np(g) * d).sum() - want) <= 1e-5 * np.abs(_np(g) * d).sum() + 1e-6 * abs(want), i


def test_repeats_streams_and_wide_offsets():
    q, k, v, do = _draw(900, 8, 2, 128, "bf16", 16)
    starts = _int([0, 500, 900])
    o, lse = pc.attention_fwd(q, k, v, starts=starts)
    first = pc.attention_bwd(q, k, v, o, lse, do, starts=starts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, l2 = pc.attention_fwd(q, k, v, starts=starts)
        again = pc.attention_bwd(q, k, v, o, lse, do, starts=starts)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o2) and torch.equal(lse, l2) and all(torch.equal(first[n], again[n]) for n in first)
    # token strides that take the last rows past 2^31 elements
    big = torch.empty((1 << 31) + (1 << 22), dtype=torch.bfloat16, device="cuda")
    far = [big.as_strided((200, 2, 64), (10790000, 64, 1), off) for off in (0, 4096, 8192, 12288)]
    near = [t[:200, :2, :64].contiguous() for t in (q, k, v, do)]
    for a, t in zip(far, near):
        a.copy_(t)
    for x in (near, far):
        o, lse = pc.attention_fwd(*x[:3])
        got = [o, lse, *pc.attention_bwd(*x[:3], o, lse, x[3]).values()]
        want = got if x is near else want
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_starts_that_are_out_of_order_fault_nothing():
    q, k, v, do = _draw(300, 2, 1, 64, "bf16", 17)
    for bad in ([0, 1000, 300], [-5, 100, 300], [200, 100, 300], [400, 500, 600], [0, 300, -1]):
        starts = _int(bad)
        o, lse = pc.attention_fwd(q, k, v, starts=starts)
        pc.attention_bwd(q, k, v, o, lse, do, starts=starts)
    torch.cuda.synchronize()


def test_empty():
    q, k, v, do = _draw(0, 4, 2, 64, "bf16", 18)
    o, lse = pc.attention_fwd(q, k, v)
    assert o.shape == q.shape and lse.shape == (4, 0)
    assert pc.attention_bwd(q, k, v, o, lse, do, starts=_int([0, 0]))["dk"].shape == k.shape
    q, k, v, do = _draw(8, 4, 2, 64, "bf16", 18)
    out = torch.full_like(q, 3.0)
    pc.attention_fwd(q, k, v, starts=_int([0]), out=out)  # no sequences
    assert (out == 3.0).all()


def test_refusals():
    q, k, v, do = _draw(8, 4, 2, 64, "bf16", 19)
    o, lse = pc.attention_fwd(q, k, v)
    with pytest.raises(ValueError, match="k has shape"):
        pc.attention_fwd(q, k[:7], v[:7])
    with pytest.raises(ValueError, match="v has shape"):
        pc.attention_fwd(q, k, v[:, :1])
    with pytest.raises(TypeError, match="v must be torch.bfloat16"):
        pc.attention_fwd(q, k, v.float())
    with pytest.raises(TypeError, match="starts must be torch.int32"):
        pc.attention_fwd(q, k, v, starts=torch.tensor([0, 8], device="cuda"))
    with pytest.raises(ValueError, match="must have 3 dimensions"):
        pc.attention_fwd(q[None], k, v)
    with pytest.raises(pc.PCError, match="multiple of the keys' heads"):
        pc.attention_fwd(q[:, :3], k, v)
    with pytest.raises(pc.PCError, match="o may not be q"):
        pc.attention_fwd(q, k, v, out=q)
    with pytest.raises(pc.PCError, match="head sizes up to"):
        pc.attention_fwd(*[torch.zeros(2, 1, 260, device="cuda")] * 3)
    with pytest.raises(ValueError, match="lse has shape"):
        pc.attention_bwd(q, k, v, o, lse[:2].contiguous(), do)
    with pytest.raises(pc.PCError, match="dv may not be dk"):
        d = torch.empty_like(k)
        pc.attention_bwd(q, k, v, o, lse, do, dk=d, dv=d)
