"""GPU parity of attention over a paged cache (pc_paged_attention) and of the cache's bookkeeping and writes
(pc_paged_plan, pc_paged_write) against float64: single tokens, chunks, pages that end inside tiles, shared and missing
pages, ranges of long caches that are joined.

Tolerances as for attention over packed sequences (tests/test_gpu_attention.py); a join of ranges adds a few
roundings to each term."""
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
    pc.device_status()


def _np(t):
    return t.detach().double().cpu().numpy()


def _int(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _cache(lengths, new, H, Hk, D, page, dtype, seed, spare=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(TYPES[dtype])  # noqa: E731
    need = [-(-n // page) for n in lengths]
    order = np.random.default_rng(seed).permutation(sum(need) + 3)
    W = max(need + [0]) + spare
    tables, at = np.full((len(lengths), W), -1), 0
    for b, n in enumerate(need):
        tables[b, :n] = order[at:at + n]
        at += n
    q = r(sum(new), H, D)
    kp, vp = (r(len(order), page, Hk, D) for _ in range(2))
    for b, n in enumerate(lengths):  # what lies behind a length is never read into an output
        if n % page:
            last = tables[b, n // page]
            kp[last, n % page:], vp[last, n % page:] = float("nan"), float("inf")
    return q, kp, vp, tables


def check(lengths, new, H, Hk, D, page, dtype, seed=1, scale=None, parts=None):
    q, kp, vp, tables = parts or _cache(lengths, new, H, Hk, D, page, dtype, seed)
    starts = np.concatenate([[0], np.cumsum(new)])
    even = len(set(new)) == 1 and seed % 2
    lse = torch.full((H, q.shape[0]), 7.0, device="cuda")
    o = pc.paged_attention(q, kp, vp, _int(tables), _int(lengths), starts=None if even else _int(starts), scale=scale, lse=lse)
    pc.device_status()
    s = D ** -0.5 if scale is None else scale
    ro, rl, size, reach = A.paged_fwd(_np(q), _np(kp), _np(vp), tables, lengths, starts, s, sizes=True)
    E, n = (D + 8) * U * reach, max(list(lengths) + [1])
    bf = dtype == "bf16"
    tol = size * (2 * E.T[..., None] + (n + 32) * U) + (2.0 ** -8 * (size + np.abs(ro)) if bf else 0) + 1e-30
    got = _np(o)
    assert np.isfinite(got).all() and np.all(np.abs(got - ro) <= tol)
    if bf:
        assert np.linalg.norm(got - ro) <= 3 * 1.7e-3 * np.linalg.norm(ro) + 1e-30
    seen = np.isfinite(rl)
    z = _np(lse)
    assert np.array_equal(np.isneginf(z), ~seen)
    assert np.all(np.abs(z - rl)[seen] <= (E + (n + 32 + 2 * np.abs(rl)) * U)[seen])
    return o


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("H,Hk,D,page", [(1, 1, 1, 1), (8, 2, 128, 16), (4, 4, 64, 16), (3, 1, 128, 5), (32, 8, 128, 16), (5, 1, 72, 7),
                                         (16, 1, 64, 64), (40, 2, 96, 48), (6, 2, 256, 32), (17, 1, 128, 128), (2, 1, 40, 300)])
def test_one_token_each(H, Hk, D, page, dtype):
    lengths = [1, 2, 15, 16, 17, 64, 65, 127, 300, 513]
    check(lengths, [1] * len(lengths), H, Hk, D, page, dtype, seed=3)
    check(lengths, [1] * len(lengths), H, Hk, D, page, dtype, seed=4)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("H,Hk,D,page", [(4, 1, 128, 16), (8, 2, 64, 32), (6, 2, 128, 13), (2, 2, 80, 64), (3, 1, 128, 256)])
@pytest.mark.parametrize("new", [[2, 2], [5, 1], [17, 3], [64, 33], [200, 129], [0, 40]])
def test_chunks(H, Hk, D, page, new, dtype):
    for past in ((0, 0), (1, 300), (127, 128), (700, 5)):
        lengths = [m + p for m, p in zip(new, past)]
        check(lengths, new, H, Hk, D, page, dtype, seed=5)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("most", [1, 3, 200])
@pytest.mark.parametrize("B,page", [(128, 16), (300, 16), (300, 13)])
def test_many_sequences(B, page, most, dtype):
    rng = np.random.default_rng(B + most)
    new = rng.integers(0, most + 1, B) * (rng.random(B) < (0.1 if most > 3 else 0.9))
    new[[5, B - 1]] = most
    check((new + rng.integers(0, 300, B)).tolist(), new.tolist(), 8, 2, 128, page, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("page", [16, 64, 100])
def test_long_caches_are_cut_and_joined(page, dtype):
    check([20001], [1], 8, 2, 128, page, dtype)
    check([9000, 1, 5003, 0], [1, 1, 1, 0], 4, 1, 64, page, dtype, seed=2)
    check([9000, 4000], [3, 40], 4, 1, 128, page, dtype, seed=2)
    check([30000], [300], 4, 2, 128, page, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [128, 40])
def test_rows_that_see_nothing(dtype, D):
    check([0, 3, 1, 0], [2, 5, 1, 0], 4, 2, D, 16, dtype, seed=6)
    check([0, 20], [300, 200], 4, 2, D, 16, dtype, seed=6)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("new", [1, 3, 100])
def test_rows_behind_the_last_sequence_stay(dtype, new):
    lengths, T = [400, 9000], 2 * new + 7
    q, kp, vp, tables = _cache(lengths, [T, 0], 4, 2, 64, 16, dtype, 7)
    out, lse = torch.full_like(q, 5.0), torch.full((4, T), 5.0, device="cuda")
    pc.paged_attention(q, kp, vp, _int(tables), _int(lengths), starts=_int([0, new, 2 * new]), out=out, lse=lse)
    assert (out[2 * new:] == 5.0).all() and (lse[:, 2 * new:] == 5.0).all() and torch.isfinite(out).all()
    assert not (out[:2 * new] == 5.0).any()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("new", [1, 4, 150])
def test_missing_pages_count_as_masked_and_are_reported(dtype, new):
    """Entries below zero, past the pages and past the table's width; the rest as if they were not there."""
    H, Hk, D, page, n = 4, 2, 128, 16, 700
    q, kp, vp, tables = _cache([n], [new], H, Hk, D, page, dtype, 8, spare=0)
    pc.device_status()
    for bad in (-1, len(kp), 2 ** 31 - 1, -2 ** 31):
        t = tables.copy()
        t[0, 3], t[0, 20] = bad, bad
        o = pc.paged_attention(q, kp, vp, _int(t), _int([n]), starts=_int([0, new]))
        with pytest.raises(pc.PCError, match="PC_ERR_RANGE.*outside the paged cache"):
            pc.device_status()
        pc.device_status()
        k, v = (_np(x) for x in (kp, vp))
        s = np.array([p for p in range(n) if p // page not in (3, 20)])
        k, v = (x[tables[0, s // page], s % page] for x in (k, v))
        want = np.concatenate([A.attend(_np(q[i:i + 1]), k[s <= n - new + i], v[s <= n - new + i], D ** -0.5, 10 ** 6)[0]
                               for i in range(new)])
        tol = 2.0 ** -7 if dtype == "bf16" else 1e-4  # (of values around one: which keys count is what is tested)
        assert np.abs(_np(o) - want).max() <= tol
    # past the width: every row sees the keys that the table holds (the rows behind the length, which _cache fills with NaN, are
    # keys then, and get finite values for it)
    k2, v2 = (torch.nan_to_num(x, nan=0.5, posinf=2.0) for x in (kp, vp))
    o = pc.paged_attention(q, k2, v2, _int(tables), _int([n + 10 ** 6]), starts=_int([0, new]))
    k, v = (_np(x)[tables[0]].reshape(-1, Hk, D) for x in (k2, v2))
    want = np.concatenate([A.attend(_np(q[i:i + 1]), k, v, D ** -0.5, 10 ** 6)[0] for i in range(new)])
    assert np.abs(_np(o) - want).max() <= tol
    with pytest.raises(pc.PCError, match="PC_ERR_RANGE"):
        pc.device_status()
    pc.paged_attention(q, kp[:0], vp[:0], _int(tables), _int([n]), starts=_int([0, new]))  # no pages at all
    with pytest.raises(pc.PCError, match="PC_ERR_RANGE"):
        pc.device_status()
    o = pc.paged_attention(q, kp, vp, _int(tables[:, :0]), _int([0]), starts=_int([0, new]))
    assert not o.any()
    pc.device_status()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("new", [1, 90])
def test_shared_pages_strides_and_streams(dtype, new):
    H, Hk, D, page, lengths = 4, 2, 64, 16, [600, 500]
    q, kp, vp, tables = _cache(lengths, [new, new], H, Hk, D, page, dtype, 9)
    tables[1, :20] = tables[0, :20]  # a prompt in common
    want = check(lengths, [new, new], H, Hk, D, page, dtype, parts=(q, kp, vp, tables))
    both = torch.empty(len(kp), Hk, page, 2 * D, dtype=q.dtype, device="cuda")  # heads first, keys beside values
    k2, v2 = both[..., :D].transpose(1, 2), both[..., D:].transpose(1, 2)
    k2.copy_(kp), v2.copy_(vp)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = pc.paged_attention(q, k2, v2, _int(tables), _int(lengths), starts=_int([0, new, 2 * new]))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    odd = [torch.empty(len(kp), page, Hk, D + 1, dtype=q.dtype, device="cuda")[..., 1:].copy_(t) for t in (kp, vp)]
    check(lengths, [new, new], H, Hk, D, page, dtype, parts=(q, *odd, tables))


def test_pages_past_32_bit_offsets():
    H, Hk, D, page, pages = 2, 1, 64, 16, 2_200_000  # 2.25e9 elements each
    kp, vp = (torch.zeros(pages, page, Hk, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    far = torch.tensor([pages - 1, pages - 7, 3, pages - 2], device="cuda")
    for t in (kp, vp):
        t[far] = torch.randn(4, page, Hk, D, generator=g, device="cuda").bfloat16()
    q = torch.randn(130, H, D, generator=g, device="cuda").bfloat16()
    near = [t[far].contiguous() for t in (kp, vp)]
    for new in (1, 130):
        n = [60 if new == 1 else 64]
        got = pc.paged_attention(q[:new], kp, vp, far[None].int(), _int(n))
        assert torch.equal(got, pc.paged_attention(q[:new], *near, _int([[0, 1, 2, 3]]), _int(n)))
    slots = torch.tensor([(pages - 1) * page + 5], device="cuda")
    row = torch.full((1, Hk, D), 2.0, dtype=torch.bfloat16, device="cuda")
    pc.paged_write(row, row * 2, kp, vp, slots)
    assert (kp[-1, 5] == 2).all() and (vp[-1, 5] == 4).all() and not (kp[-1, 4] == 2).any()


@pytest.mark.parametrize("B,W,page,short", [(1, 3, 4, 0), (5, 6, 16, 0), (40, 9, 7, 0), (40, 9, 7, 11), (1500, 4, 16, 0),
                                            (1024, 3, 1, 5), (2100, 5, 64, 0)])
def test_plan(B, W, page, short):
    rng = np.random.default_rng(B + W)
    cached = rng.integers(0, W * page, B)
    added = np.minimum(rng.integers(0, 2 * page + 2, B) * (rng.random(B) < 0.7), W * page - cached)
    cached[B // 2], added[0] = 0, 0
    need = (-(-(cached + added) // page) + -cached // page).sum()
    ids = rng.permutation(10 ** 6)
    tables = np.full((B, W), -1)
    for b in range(B):
        tables[b, :-(-cached[b] // page)] = ids[b * W:b * W + -(-cached[b] // page)]
    free = ids[B * W:][:max(int(need) - short, 0)]
    T = int(added.sum())
    dev = _int(tables)
    want = A.paged_plan(cached, added, tables, free, page, T)
    for again in range(2):  # planned twice: the same
        got = pc.paged_plan(_int(cached), _int(added), dev, _int(free), page, T)
        for n in ("starts", "lengths", "positions", "slots", "taken"):
            assert np.array_equal(got[n].cpu().numpy(), want[n]), n
        assert np.array_equal(dev.cpu().numpy(), want["tables"]) and got["slots"].dtype == torch.int64


def test_plan_at_the_ends():
    # values below zero count as none; tokens past the table's width and behind the last request have no place
    args = ([-3, 30, 5], [2, 8, -4], [[-1, -1], [4, 5], [6, -1]], [9, 8], 16, 14)
    dev = _int(args[2])
    got = pc.paged_plan(*[_int(x) for x in args[:2]], dev, _int(args[3]), *args[4:])
    want = A.paged_plan(*args)
    for n in ("starts", "lengths", "positions", "slots", "taken"):
        assert np.array_equal(got[n].cpu().numpy(), want[n]), n
    assert np.array_equal(dev.cpu().numpy(), want["tables"]) and want["slots"].tolist()[-10:] == [-1] * 10
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    got = pc.paged_plan(empty, empty, empty.reshape(0, 4), empty, 16, 3)
    assert got["starts"].tolist() == [0] and got["taken"].tolist() == [0] and got["slots"].tolist() == [-1] * 3
    huge = _int([2 ** 31 - 1] * 3)  # sums that overflow: nothing meaningful, and nothing out of range
    pc.paged_plan(huge, huge, _int([[1, 2]] * 3), _int([3]), 16, 100)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("Hk,D,page", [(1, 1, 1), (2, 64, 16), (3, 40, 7), (8, 128, 64), (1, 257, 4)])
def test_write(Hk, D, page, dtype):
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(TYPES[dtype])  # noqa: E731
    P, T = 9, min(2 * page + 1, 9 * page)
    proj = r(T, 3 * Hk * D)
    k, v = (proj[:, i * Hk * D:(i + 1) * Hk * D].unflatten(-1, (Hk, D)) for i in (1, 2))
    kp, vp = r(P, page, Hk, D), r(P, Hk, page, D).transpose(1, 2)
    slots = torch.randperm(P * page, device="cuda")[:T]
    slots[0] = -1
    want = []
    for t, x in ((kp, k), (vp, v)):
        w = t.clone().flatten(0, 1)
        w[slots[1:]] = x[1:]
        want.append(w.unflatten(0, (P, page)))
    pc.paged_write(k, v, kp, vp, slots)
    pc.device_status()
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    slots[1:] = P * page
    slots[-1] = 2 ** 62
    pc.paged_write(k, v, kp, vp, slots)
    if T > 1:
        with pytest.raises(pc.PCError, match="PC_ERR_RANGE"):
            pc.device_status()
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("H,Hk,D", [(4, 2, 128), (6, 2, 40)])
def test_a_prompt_then_chunks_then_tokens(H, Hk, D, dtype):
    """Planned, turned, written and read step by step: the rows of the whole sequences' attention."""
    page, B, W = 16, 3, 24
    g = torch.Generator(device="cuda").manual_seed(3)
    steps = [[70, 5, 0], [1, 1, 1], [130, 0, 40], [1, 1, 1], [1, 1, 1]]
    total = np.sum(steps, 0)
    xs = [[torch.randn(int(n), h, D, generator=g, device="cuda").to(TYPES[dtype]) for h in (H, Hk, Hk)] for n in total]
    f, _ = pc.rotary_frequencies(D)
    w = [1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    kp, vp = (torch.full((80, page, Hk, D), float("nan"), dtype=TYPES[dtype], device="cuda") for _ in range(2))
    tables, free = _int(np.full((B, W), -1)), torch.randperm(80, device="cuda").int()
    lengths, done, outs = _int([0] * B), [0] * B, [[] for _ in range(B)]
    for new in steps:
        q, k, v = (torch.cat([xs[b][i][done[b]:done[b] + new[b]] for b in range(B)]) for i in range(3))
        plan = pc.paged_plan(lengths, _int(new), tables, free, page, sum(new))
        q, k = pc.qk_norm_rotary_fwd(q, k, plan["positions"], f, *w)
        pc.paged_write(k, v, kp, vp, plan["slots"])
        o = pc.paged_attention(q, kp, vp, tables, plan["lengths"], starts=plan["starts"])
        lengths, free = plan["lengths"], free[int(plan["taken"]):].contiguous()
        for b, part in enumerate(o.split(new)):
            outs[b].append(part)
            done[b] += new[b]
    pc.device_status()
    for b in range(B):
        pos = torch.arange(done[b], device="cuda", dtype=torch.int32)
        q, k = pc.qk_norm_rotary_fwd(xs[b][0], xs[b][1], pos, f, *w)
        want, _ = pc.attention_fwd(q, k, xs[b][2])
        got = torch.cat(outs[b])
        ro, _, size, reach = A.packed_fwd(_np(q), _np(k), _np(xs[b][2]), [0, done[b]], D ** -0.5, sizes=True)
        tol = size * (2 * (D + 8) * U * reach.T[..., None] + (done[b] + 32) * U)
        tol = tol + (2.0 ** -8 * (size + np.abs(ro)) if dtype == "bf16" else 0)
        assert np.all(np.abs(_np(got) - ro) <= tol) and np.all(np.abs(_np(want) - ro) <= tol)


def test_captured_steps_replay_with_new_lengths():
    """A step's plan, writes and attention in one graph: the lengths are read when it is replayed."""
    H, Hk, D, page, B, W = 4, 2, 128, 16, 3, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    kp, vp = (torch.randn(200, page, Hk, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    x = [torch.randn(B, h, D, generator=g, device="cuda").bfloat16() for h in (H, Hk, Hk)]
    tables, free = torch.randperm(192, device="cuda").int().reshape(B, W), torch.arange(192, 200, device="cuda").int()
    cached, added = _int([5, 900, 100]), _int([1] * B)

    def step():
        plan = pc.paged_plan(cached, added, tables, free, page, B)
        pc.paged_write(x[1], x[2], kp, vp, plan["slots"])
        return pc.paged_attention(x[0], kp, vp, tables, plan["lengths"], starts=plan["starts"])

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for n in ([5, 900, 100], [1, 1, 40], [1000, 0, 17]):
        cached.copy_(_int(n))
        out.fill_(float("nan"))
        graph.replay()
        got = out.clone()
        assert torch.equal(got, step()) and torch.isfinite(got).all()
    pc.device_status()


def test_empty_and_refusals():
    q, kp, vp, tables = _cache([20, 30], [1, 1], 4, 2, 64, 16, "bf16", 10)
    t, n = _int(tables), _int([20, 30])
    assert pc.paged_attention(q[:0], kp, vp, t, n, starts=_int([0, 0, 0])).shape == (0, 4, 64)
    with pytest.raises(ValueError, match="tables has shape"):
        pc.paged_attention(q, kp, vp, t[:1].contiguous(), n)
    with pytest.raises(ValueError, match="starts has shape"):
        pc.paged_attention(q, kp, vp, t, n, starts=_int([0, 2]))
    with pytest.raises(ValueError, match="v_pages has shape"):
        pc.paged_attention(q, kp, vp[:3], t, n)
    with pytest.raises(ValueError, match="head size"):
        pc.paged_attention(q[..., :32], kp, vp, t, n)
    with pytest.raises(TypeError, match="k_pages must be torch.bfloat16"):
        pc.paged_attention(q, kp.float(), vp, t, n)
    with pytest.raises(pc.PCError, match="multiple of B"):
        pc.paged_attention(torch.cat([q, q[:1]]), kp, vp, t, n)
    with pytest.raises(TypeError, match="added must be torch.int32"):
        pc.paged_plan(n, n.long(), t, n, 16, 2)
    with pytest.raises(pc.PCError, match="page_size"):
        pc.paged_plan(n, n, t, n, 0, 2)
    with pytest.raises(TypeError, match="slots must be torch.int64"):
        pc.paged_write(kp[0], vp[0], kp, vp, n)


def test_heads_without_features_are_refused():
    x, t, n = torch.zeros(2, 1, 0, device="cuda"), _int([[0], [0]]), _int([1, 1])
    with pytest.raises(pc.PCError, match="head size must be >= 1"):
        pc.attention_fwd(x, x, x)
    with pytest.raises(pc.PCError, match="head size must be >= 1"):
        pc.paged_attention(x, x[:, None], x[:, None], t, n)
