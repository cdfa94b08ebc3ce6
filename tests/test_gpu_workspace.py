"""Calls that must not meet in scratch memory: host threads on one stream, a graph and the
larger calls after its capture, two graphs at a time. Equal bits throughout."""
import threading

import pytest
import torch

import log_space_sum_gb300 as pc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pc.load()


def _cases(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    G, x, dy, w = r(2, 200, 330), r(400, 256), r(400, 256), r(256)
    q, k, v, do = (r(2, 700, 2, 64).bfloat16() for _ in range(4))
    decay, n = -torch.rand(2, generator=g, device="cuda"), torch.tensor([120, 60], dtype=torch.int32, device="cuda")
    _, mean, rstd = pc.layer_norm_fwd(x, w)
    return [lambda: [pc.orthogonalize(G)], lambda: [pc.orthogonalize(G, precision="fp32")],
            lambda: pc.layer_norm_bwd(dy, x, w, mean, rstd), lambda: pc.linear_attention_fwd(q, k, v, decay),
            lambda: pc.linear_attention_fwd(q, k, v, decay, lengths=n),  # one chunk each: no segment waits
            lambda: pc.linear_attention_bwd(q, k, v, decay, do).values()]


def test_threads_on_one_stream():
    mine, theirs = _cases(1), _cases(2)
    want = [[[t.clone() for t in fn()] for fn in cases] for cases in (mine, theirs)]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(2)

    def work(cases, wanted, order):
        start.wait()
        for i in range(20):
            for c in order[i % len(order):] + order[:i % len(order)]:
                got = list(cases[c]())
                wrong.extend(~torch.stack([(a == b).all() for a, b in zip(got, wanted[c])]).all().reshape(1))

    n = list(range(len(mine)))
    threads = [threading.Thread(target=work, args=(mine, want[0], n)),
               threading.Thread(target=work, args=(theirs, want[1], n[::-1]))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    pc.device_status()
    assert len(wrong) == 2 * 20 * len(n) and not torch.stack(wrong).any()


def _graph(fn, stream):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        out = list(fn())
    return g, out


def test_a_larger_call_between_capture_and_replay():
    s = torch.cuda.Stream()
    for fn in _cases(3):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            want = [t.clone() for t in fn()]  # warm, on the stream that is captured
        torch.cuda.synchronize()
        g, out = _graph(fn, s)
        with torch.cuda.stream(s):
            pc.orthogonalize(torch.randn(1, 2000, 2000, device="cuda"))  # a larger workspace takes the place of the warm one
            others = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
        torch.cuda.synchronize()
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))
        assert all(bool((t == 7).all()) for t in others)


def test_two_graphs_at_a_time():
    for a, b in zip(_cases(4), _cases(5)):
        want = [[t.clone() for t in fn()] for fn in (a, b)]
        torch.cuda.synchronize()
        graphs = [_graph(fn, None) for fn in (a, b)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(20):
            for (g, _), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        pc.device_status()
        for w, (_, out) in zip(want, graphs):
            assert all(torch.equal(x, y) for x, y in zip(w, out))
