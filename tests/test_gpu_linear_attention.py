"""GPU parity of linear attention (pc_linear_attention_fwd / _bwd / _step) against the
float64 recurrences: head sizes on both sides of the tensor-core variant's limits, lengths
of zero, one and past several tiles, states, strides, decays of one and zero.

Tolerances. u = 2^-24. Every output is a sum of products; with the oracle run on absolute
values as its size, the float32 path may be off by u for each rounding that a term passes:
the sums over a head (Dk or Dv), over a tile and over the tiles, and the decay's exponential
(a few u of a power, whose exponent log_decay n carries u |log_decay| n). With bf16 elements each
term passes at most one rounding to bf16 (2^-8 at most: of a score, or of the state that is
read) and the output one more; as these roundings are independent, the 2-norm of the
error is three times 1.7e-3 (a bf16 rounding's root mean square) at most. The state is held
in float32 and passes no bf16 rounding."""
import numpy as np
import pytest
import torch

import log_space_sum_gb300 as pc
from oracle import factor_network as F

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pc.load()


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _draw(B, T, H, dk, dv, dtype, seed, state=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k = (r(B, T, H, dk).to(TYPES[dtype]) for _ in range(2))
    v, do = (r(B, T, H, dv).to(TYPES[dtype]) for _ in range(2))
    decay = -torch.exp2(-1 - 7 * torch.rand(H, generator=g, device="cuda"))
    S, dS = (r(B, H, dk, dv) if state else None for _ in range(2))
    return q, k, v, do, decay, S, dS


def _close(got, want, size, terms, bf16, what):
    got = _np(got)
    assert np.isfinite(got).all(), what
    tol = terms * U * size + 1e-30
    if bf16:
        tol = tol + 2.0 ** -8 * size + 2.0 ** -8 * np.abs(want)
        norm = np.linalg.norm(want)
        assert np.linalg.norm(got - want) <= 3 * 1.7e-3 * norm + 1e-30, what
    assert np.all(np.abs(got - want) <= tol), what


def _terms(dk, dv, T, decay, state):
    g = np.abs(_np(decay))
    g = g[np.isfinite(g)]
    return max(dk, dv) + 128 + T // 32 + 16 + 4 * (1 + (g.max() if g.size else 0) * min(T, 128))


def _check(q, k, v, do, decay, S, dS, dtype, scale=0.3, lengths=None, **out):
    bf16 = dtype == "bf16"
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    Q, K, V, G, D, S0, E = (_np(t) for t in (q, k, v, do, decay, S, dS))
    terms = _terms(q.shape[-1], v.shape[-1], q.shape[1], decay, S)
    mag = lambda *ts: [None if t is None else np.abs(t) for t in ts]  # noqa: E731
    o, state = pc.linear_attention_fwd(q, k, v, decay, scale=scale, state=S, lengths=n)
    ln = None if lengths is None else np.array(lengths)
    ro, rs = F.linear_attention_fwd(Q, K, V, D, scale, S0, ln)
    aq, ak, av, ag, as0, ae = mag(Q, K, V, G, S0, E)
    zo, zs = F.linear_attention_fwd(aq, ak, av, D, scale, as0, ln)
    _close(o, ro, zo, terms, bf16, "o")
    _close(state, rs, zs, terms, False, "state")
    got = pc.linear_attention_bwd(q, k, v, decay, do, scale=scale, state=S, dstate=dS, lengths=n, **out)
    want = F.linear_attention_bwd(Q, K, V, D, G, scale, S0, E, ln)
    size = F.linear_attention_bwd(aq, ak, av, D, ag, scale, as0, ae, ln)
    for name, w, z in zip(("dq", "dk", "dv", "dstate"), want, size):
        _close(got[name], w, z, terms, bf16 and name != "dstate", name)
    return o, state, got


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,T,H,dk,dv", [
    (1, 1, 1, 1, 1), (2, 1, 3, 128, 128), (1, 5, 2, 3, 9), (2, 33, 2, 64, 64), (1, 127, 2, 128, 64),
    (1, 128, 2, 64, 128), (2, 129, 3, 128, 128), (1, 300, 2, 40, 72), (1, 257, 1, 120, 8), (1, 90, 2, 200, 136),
    (1, 40, 1, 256, 256), (1, 1000, 2, 128, 128), (1, 70, 3, 12, 100)])
@pytest.mark.parametrize("state", [False, True])
def test_sizes(B, T, H, dk, dv, dtype, state):
    _check(*_draw(B, T, H, dk, dv, dtype, B + T + dk + dv, state), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lengths", [[300, 0, 1, 129], [0, 0, 0, 0], [128, 127, 299, 256]])
def test_lengths_and_what_lies_past_them(dtype, lengths):
    q, k, v, do, decay, S, dS = _draw(4, 300, 2, 64, 128, dtype, 11)
    clean = _check(q, k, v, do, decay, S, dS, dtype, lengths=lengths)
    for b, n in enumerate(lengths):  # nothing past a length is read
        for t in (q, k, v, do):
            t[b, n:] = float("nan")
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o, state = pc.linear_attention_fwd(q, k, v, decay, scale=0.3, state=S, lengths=n)
    got = pc.linear_attention_bwd(q, k, v, decay, do, scale=0.3, state=S, dstate=dS, lengths=n)
    assert torch.equal(o, clean[0]) and torch.equal(state, clean[1])
    for name, t in got.items():
        assert torch.equal(t, clean[2][name]), name
    for b, m in enumerate(lengths):
        assert not any(t[b, m:].any() for t in (o, got["dq"], got["dk"], got["dv"]))
        if m == 0:
            assert torch.equal(state[b], S[b]) and torch.equal(got["dstate"][b], dS[b])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("value", [0.0, -float("inf"), -30.0])
def test_decays_at_the_ends(dtype, value):
    q, k, v, do, decay, S, dS = _draw(2, 200, 2, 64, 64, dtype, 12)
    decay[0] = value
    o, state, _ = _check(q, k, v, do, decay, S, dS, dtype)
    if value == -float("inf"):  # only the token itself counts
        own = (_np(q) * _np(k)).sum(-1)[..., None] * _np(v) * 0.3
        np.testing.assert_allclose(_np(o)[:, :, 0], own[:, :, 0], rtol=2 ** -6, atol=1e-5)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("layout", ["projection", "heads first", "unaligned"])
def test_strides(dtype, layout):
    B, T, H, d = 2, 150, 3, 64
    q, k, v, do, decay, S, dS = _draw(B, T, H, d, d, dtype, 13)
    want = _check(q, k, v, do, decay, S, dS, dtype)
    dt, out = TYPES[dtype], {}
    if layout == "projection":  # q, k, v and their gradients are slices of one matrix each
        cut = lambda p: [p[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(3)]  # noqa: E731
        parts = cut(torch.empty(B, T, 3 * H * d, device="cuda", dtype=dt))
        grads = cut(torch.empty(B, T, 3 * H * d, device="cuda", dtype=dt))
        out = dict(zip(("dq", "dk", "dv"), grads))
    elif layout == "heads first":
        parts = [torch.empty(B, H, T, d, device="cuda", dtype=dt).transpose(1, 2) for _ in range(3)]
    else:
        parts = [torch.empty(B, T, H, d + 1, device="cuda", dtype=dt)[..., 1:] for _ in range(3)]
    for p, t in zip(parts, (q, k, v)):
        p.copy_(t)
    got = _check(*parts, do, decay, S, dS, dtype, **out)
    if layout != "unaligned":  # the same variant: the same bits
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert all(torch.equal(got[2][n], want[2][n]) for n in want[2])
    # one value of k and v for every head, without a copy
    shared = [t[:, :, :1].expand(-1, -1, H, -1) for t in (k, v)]
    _check(q, *shared, do, decay, S, dS, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_a_prompt_then_single_tokens(dtype):
    """The recurrent form continues the chunked one."""
    B, T, H, dk, dv = 3, 140, 4, 64, 128
    q, k, v, _, decay, S, _ = _draw(B, T, H, dk, dv, dtype, 14)
    ro, rs = F.linear_attention_fwd(*(_np(t) for t in (q, k, v, decay)), 0.5, _np(S))
    zo, zs = F.linear_attention_fwd(*(np.abs(_np(t)) for t in (q, k, v)), _np(decay), 0.5, np.abs(_np(S)))
    terms = _terms(dk, dv, T, decay, S)
    o, state = pc.linear_attention_fwd(q[:, :133], k[:, :133], v[:, :133], decay, scale=0.5, state=S)
    rest = [pc.linear_attention_step(q[:, t], k[:, t], v[:, t], decay, state, scale=0.5) for t in range(133, T)]
    _close(torch.cat([o, torch.stack(rest, 1)], 1), ro, zo, terms, dtype == "bf16", "o")
    _close(state, rs, zs, terms, False, "state")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,H,dk,dv", [(1, 1, 1, 1), (3, 2, 5, 7), (2, 3, 64, 64), (5, 2, 128, 128), (2, 1, 256, 256),
                                       (2, 2, 128, 36), (1, 2, 33, 130), (700, 1, 16, 8)])
def test_step(B, H, dk, dv, dtype):
    q, k, v, _, decay, S, _ = _draw(B, 1, H, dk, dv, dtype, 15)
    decay[0] = -float("inf") if B == 3 else decay[0]
    ro, rs = F.linear_attention_fwd(*(_np(t) for t in (q, k, v, decay)), 0.5, _np(S))
    zo, zs = F.linear_attention_fwd(*(np.abs(_np(t)) for t in (q, k, v)), _np(decay), 0.5, np.abs(_np(S)))
    o = pc.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], decay, S, scale=0.5)
    _close(o, ro[:, 0], zo[:, 0], dk + 16, dtype == "bf16", "o")
    _close(S, rs, zs, 8, False, "state")


def test_long_sequence_state_and_segments():
    """Thousands of tokens of few heads: the sequence is cut over the GPU and joined; a
    decay of one makes every token count to the end."""
    q, k, v, do, decay, S, dS = _draw(1, 5000, 2, 128, 64, "bf16", 16)
    decay[1] = 0.0
    _check(q, k, v, do, decay, S, dS, "bf16")


@pytest.mark.parametrize("lengths", [None, [1500, 1499, 700, 1]])
def test_two_uneven_segments(lengths):
    """Heads for half the SMs: a long first segment beside its states' launch and a short one
    after it, in order of time (forward) and against it (in the gradient's passes where fewer
    heads leave the same room)."""
    q, k, v, do, decay, S, dS = _draw(4, 1500, 16, 64, 128, "bf16", 17)
    _check(q, k, v, do, decay, S, dS, "bf16", lengths=lengths)
    q, k, v, do, decay, S, dS = _draw(4, 1500, 6, 128, 128, "bf16", 18)
    _check(q, k, v, do, decay, S, dS, "bf16", lengths=lengths)


def test_repeats_streams_and_wide_offsets():
    q, k, v, do, decay, S, dS = _draw(2, 500, 4, 128, 128, "bf16", 17)
    first = pc.linear_attention_bwd(q, k, v, decay, do, state=S, dstate=dS)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = pc.linear_attention_bwd(q, k, v, decay, do, state=S, dstate=dS)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(first[n], again[n]) for n in first)
    # token strides that take the last rows past 2^31 elements
    big = torch.empty((1 << 31) + (1 << 22), dtype=torch.bfloat16, device="cuda")
    far = [big.as_strided((1, 200, 2, 64), (0, 10790000, 64, 1), off) for off in (0, 4096, 8192)]
    near = [t[:1, :200, :2, :64].contiguous() for t in (q, k, v)]
    for a, t in zip(far, near):
        a.copy_(t)
    want, got = (pc.linear_attention_fwd(*x, decay[:2].contiguous()) for x in (near, far))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_empty():
    q, k, v, do, decay, S, dS = _draw(2, 0, 3, 64, 64, "bf16", 18)
    o, state = pc.linear_attention_fwd(q, k, v, decay, state=S)
    assert o.shape == v.shape and torch.equal(state, S)
    got = pc.linear_attention_bwd(q, k, v, decay, do, state=S, dstate=dS)
    assert torch.equal(got["dstate"], dS)
    none = [t[:0] for t in (q, k, v)]
    assert pc.linear_attention_fwd(*none, decay)[1].shape == (0, 3, 64, 64)


def test_refusals():
    q, k, v, do, decay, S, dS = _draw(2, 8, 3, 64, 64, "bf16", 19)
    with pytest.raises(ValueError, match="k has shape"):
        pc.linear_attention_fwd(q, k[:, :7], v, decay)
    with pytest.raises(TypeError, match="v must be torch.bfloat16"):
        pc.linear_attention_fwd(q, k, v.float(), decay)
    with pytest.raises(ValueError, match="log_decay has shape"):
        pc.linear_attention_fwd(q, k, v, decay[:2])
    with pytest.raises(ValueError, match="state has shape"):
        pc.linear_attention_fwd(q, k, v, decay, state=S[:, :, :32].contiguous())
    with pytest.raises(TypeError, match="lengths must be torch.int32"):
        pc.linear_attention_fwd(q, k, v, decay, lengths=torch.ones(2, device="cuda", dtype=torch.int64))
    with pytest.raises(ValueError, match="contiguous along its last"):
        pc.linear_attention_fwd(q.transpose(-1, -2).contiguous().transpose(-1, -2), k, v, decay)
    with pytest.raises(ValueError, match="do has shape"):
        pc.linear_attention_bwd(q, k, v, decay, do[..., :32])
    with pytest.raises(TypeError, match="state must be"):
        pc.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], decay, None)
    with pytest.raises(pc.PCError, match="state_out may not be state"):
        pc.linear_attention_fwd(q, k, v, decay, state=S, state_out=S)
    wide = torch.zeros(1, 2, 1, 300, device="cuda")
    with pytest.raises(pc.PCError, match="head sizes up to"):
        pc.linear_attention_fwd(wide, wide, wide, decay[:1])
