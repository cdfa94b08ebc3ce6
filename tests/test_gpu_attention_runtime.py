"""Softmax attention, the norms with rotation and the paged cache in a program's hands: captured graphs, host threads on
one stream, waits that run out, what the profiler records, scratch of exactly the promised size. Equal bits throughout."""
import ctypes as C
import threading

import pytest
import torch

import log_space_sum_gb300 as pc
from log_space_sum_gb300 import _native as N

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pc.load()
    pc.device_status()
    yield
    pc.set_wait_limit_ns(0)


def _cases(seed, dtype="bf16", D=128):
    """Every call, in each of its variants: [(name, function of no arguments -> tensors)]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(TYPES[dtype])  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    T, H, Hk = 900, 4, 2
    q, k, v, do = r(T, H, D), r(T, Hk, D), r(T, Hk, D), r(T, H, D)
    starts, pos, (f, _) = i32([0, 500, 500, 900]), torch.arange(T, device="cuda", dtype=torch.int32), pc.rotary_frequencies(D)
    w = [torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    o, lse = pc.attention_fwd(q, k, v, starts=starts)
    kp, vp = r(200, 16, Hk, D), r(200, 16, Hk, D)
    tables, lengths = torch.randperm(200, generator=g, device="cuda").int()[:192].reshape(3, 64), i32([1000, 7, 600])
    one, some, many = i32([0, 1, 2, 3]), i32([0, 3, 3, 6]), i32([0, 200, 200, 500])
    cached, added, free = i32([5, 900, 100]), i32([1, 90, 20]), torch.arange(192, 200, device="cuda").int()

    def plan():
        t = tables.clone()
        got = pc.paged_plan(cached, added, t, free, 16, 111)
        a, b = kp.clone(), vp.clone()
        pc.paged_write(k[:111], v[:111], a, b, got["slots"])
        return [t, a, b, *got.values()]

    return [("rotary", lambda: pc.qk_norm_rotary_fwd(q, k, pos, f, *w)),
            ("rotary gradient", lambda: pc.qk_norm_rotary_bwd(do, k, q, k, pos, f, *w).values()),
            ("attention", lambda: pc.attention_fwd(q, k, v, starts=starts)),
            ("attention gradient", lambda: pc.attention_bwd(q, k, v, o, lse, do, starts=starts).values()),
            ("one token each", lambda: [pc.paged_attention(q[:3], kp, vp, tables, lengths, starts=one)]),
            ("a few tokens", lambda: [pc.paged_attention(q[:6], kp, vp, tables, lengths, starts=some)]),
            ("chunks", lambda: [pc.paged_attention(q[:500], kp, vp, tables, lengths, starts=many)]),
            ("plan and writes", plan)]


def _took(fn):
    return [t.clone() for t in fn()]


def _same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("fp32", 40)])
def test_captured_and_replayed(dtype, D):
    for name, fn in _cases(1, dtype, D):
        want = _took(fn)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = list(fn())
        for _ in range(2):
            for t in out:
                t.zero_() if not t.is_floating_point() else t.fill_(float("nan"))
            graph.replay()
            assert _same(out, want), name
        again = _took(fn)  # a call of the stream between the graph's replays
        graph.replay()
        assert _same(out, want) and _same(again, want), name


def test_two_graphs_at_a_time():
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for (name, fn), (_, other) in zip(_cases(2), _cases(3)[::-1]):
        want, theirs = _took(fn), _took(other)
        torch.cuda.synchronize()
        graphs = []
        for f, s in ((fn, a), (other, b)):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                out = list(f())
            graphs.append((g, out))
        for _ in range(5):
            for (g, _), s in zip(graphs, (a, b)):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert _same(graphs[0][1], want) and _same(graphs[1][1], theirs), name


def test_threads_on_one_stream():
    mine, theirs = _cases(4), _cases(5)
    want = [[_took(fn) for _, fn in cases] for cases in (mine, theirs)]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(2)

    def work(cases, wanted, order):
        start.wait()
        for _ in range(10):
            for c in order:
                got = list(cases[c][1]())
                wrong.append(~torch.stack([(x == y).all() for x, y in zip(got, wanted[c])]).all().reshape(1))

    n = list(range(len(mine)))
    threads = [threading.Thread(target=work, args=(mine, want[0], n)), threading.Thread(target=work, args=(theirs, want[1], n[::-1]))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    pc.device_status()
    assert len(wrong) == 2 * 10 * len(n) and not torch.cat(wrong).any()


@pytest.mark.parametrize("D,pack", [(128, 8), (64, 1), (128, 3)])
def test_waits_that_run_out(D, pack):
    """With a limit of 1 ns the waits for products give up, the roles that this starves run into the default of 2 s, the timeout
    is reported, and with the default limit back the call gives the bits that it gave before."""
    g = torch.Generator(device="cuda").manual_seed(6)
    T, Hk = 2000, 2
    r = lambda h: torch.randn(T, h, D, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v, do = r(Hk * pack), r(Hk), r(Hk), r(Hk * pack)
    o, lse = pc.attention_fwd(q, k, v)
    kp, vp = (t.reshape(125, 16, Hk, D).contiguous() for t in (k, v))
    tables, lengths = torch.arange(125, device="cuda").int()[None], torch.tensor([T], dtype=torch.int32, device="cuda")
    for run in (lambda: pc.attention_fwd(q, k, v), lambda: pc.attention_bwd(q, k, v, o, lse, do).values(),
                lambda: [pc.paged_attention(q[:400], kp, vp, tables, lengths)]):
        want = _took(run)
        pc.device_status()
        pc.set_wait_limit_ns(1)
        try:
            run()
            torch.cuda.synchronize()
        finally:
            pc.set_wait_limit_ns(0)
        with pytest.raises(pc.PCError) as ei:
            pc.device_status()
        assert ei.value.status == 8, ei.value  # PC_ERR_TIMEOUT
        pc.device_status()  # the read cleared it
        assert _same(_took(run), want)
        pc.device_status()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_what_the_profiler_records(dtype):
    """One record of a call of attention, without flops: the lengths are on the device; none of what is no contraction."""
    for name, fn in _cases(7, dtype):
        fn()
        torch.cuda.synchronize()
        pc.profile_start(64)
        try:
            fn()
        finally:
            got = pc.profile_stop(64)
        if name.startswith("rotary") or name.startswith("plan"):
            assert got == [], name
        else:
            [(kind, ms, flops, launches)] = got
            assert kind == "attention" and flops == 0 and 1 <= launches <= 4 and 0 < ms < 1000, name


@pytest.mark.parametrize("shift", [0, 16])
def test_scratch_of_the_promised_size(shift):
    """Nothing outside it is written, wherever it starts."""
    lib, guard = N.load(), 4096
    stream = torch.cuda.current_stream().cuda_stream
    g = torch.Generator(device="cuda").manual_seed(8)

    def around(nbytes, call):
        all_ = torch.full((2 * guard + shift + nbytes,), 0xA5, dtype=torch.uint8, device="cuda")
        first = guard + shift
        assert call(C.c_void_p(all_.data_ptr() + first), nbytes) == 0, lib.pc_last_error()
        torch.cuda.synchronize()
        assert (all_[:first] == 0xA5).all() and (all_[first + nbytes:] == 0xA5).all()

    ll = lambda *v: (C.c_longlong * len(v))(*v)  # noqa: E731
    p = lambda t: C.c_void_p(t.data_ptr())  # noqa: E731
    nb = C.c_size_t(0)
    for dt, code in ((torch.float32, 0), (torch.bfloat16, 1)):
        for H, Hk, D, new in ((4, 2, 128, 1), (6, 3, 64, 2), (8, 1, 72, 37), (5, 1, 40, 300)):
            r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
            q, kp, vp, n = r(2 * new, H, D), r(300, 32, Hk, D), r(300, 32, Hk, D), torch.tensor([4700, 900], device="cuda").int()
            tables, o = torch.randperm(300, device="cuda").int().reshape(2, 150), torch.empty(2 * new, H, D, dtype=dt, device="cuda")
            want = pc.paged_attention(q, kp, vp, tables, n)
            assert lib.pc_paged_attention_workspace(2, 2 * new, H, Hk, D, 300, 32, 150, code, C.byref(nb)) == 0
            st = ll(H * D, D, 32 * Hk * D, Hk * D, D, 32 * Hk * D, Hk * D, D, H * D, D)
            around(nb.value, lambda ws, size: lib.pc_paged_attention(2, 2 * new, H, Hk, D, 300, 32, 150, p(q), p(kp), p(vp), st,
                                                                    p(tables), p(n), None, D ** -0.5, p(o), None, code, ws, size, stream))
            assert torch.equal(o, want)
            T = 301
            q, k, v, do = r(T, H, D), r(T, Hk, D), r(T, Hk, D), r(T, H, D)
            o, lse = pc.attention_fwd(q, k, v)
            want = pc.attention_bwd(q, k, v, o, lse, do)
            got = [torch.empty_like(t) for t in (q, k, v)]
            assert lib.pc_attention_bwd_workspace(1, T, H, Hk, D, code, C.byref(nb)) == 0
            st = ll(*([H * D, D] + [Hk * D, D] * 2 + [H * D, D] * 3 + [Hk * D, D] * 2))
            around(nb.value, lambda ws, size: lib.pc_attention_bwd(1, T, H, Hk, D, p(q), p(k), p(v), p(o), p(do), st, None, D ** -0.5,
                                                                  p(lse), *[p(t) for t in got], code, ws, size, stream))
            assert _same(got, list(want.values()))
    T, H, Hk, D = 700, 4, 2, 128
    q, k, w = r(T, H, D), r(T, Hk, D), [torch.empty(D, device="cuda") for _ in range(2)]
    got = [torch.empty_like(q), torch.empty_like(k)]
    want = pc.qk_norm_rotary_bwd(q, k, q, k)
    assert lib.pc_qk_norm_rotary_bwd_workspace(T, H, Hk, D, 1, C.byref(nb)) == 0
    st = ll(*([H * D, D, Hk * D, D] * 3))
    around(nb.value, lambda ws, size: lib.pc_qk_norm_rotary_bwd(T, H, Hk, D, 0, p(q), p(k), p(q), p(k), st, None, None, None, None,
                                                               1e-6, 1.0, 0, 1, *[p(t) for t in got], *[p(t) for t in w], 0, code, ws,
                                                               size, stream))
    assert _same(got + w, list(want.values()))
