"""The factor network's operators together: the example trains and serves, its gradient agrees
with differences of the circuit's log-likelihood, and every entry point can be captured into
a CUDA graph (bit-identical replays)."""
import os
import sys

import pytest
import torch

import log_space_sum_gb300 as pc

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import factor_network as X  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pc.load()


def test_example_trains_and_serves():
    lls, off = X.main()
    assert sum(lls[-5:]) / 5 > sum(lls[:5]) / 5 + 5  # nats a sequence of 24 tokens
    # factors of order one from bf16 activations: a few units of 2^-8 through four layers
    assert off < 0.1


@pytest.mark.parametrize("name", ["qkv", "out", "fa", "fb", "emb"])
def test_gradient_by_differences(name):
    """float32 activations and products: d(sum of ll) along the gradient's direction."""
    vocab, latents, rank = 12, 32, 3
    tokens, circuit = X.toy(8, 9, vocab, 3), X.make_circuit(vocab, latents, 4)
    net = X.FactorNetwork(vocab, latents, rank, width=32, dtype=torch.float32, seed=5)

    def ll():
        (FA, FB), saved = net.forward(tokens)
        r = pc.hmm_lowrank_fwd_bwd(tokens, circuit["pi"], circuit["A"], circuit["E"], FA, FB, precision="fp32")
        return r["ll"].sum().item(), saved, r

    _, saved, r = ll()
    grad = net.backward(saved, r["dFA"], r["dFB"])[name]
    u, eps = grad / grad.norm(), 0.05
    net.p[name] += eps * u
    up = ll()[0]
    net.p[name] -= 2 * eps * u
    down = ll()[0]
    want = grad.norm().item()
    # the central difference is off by eps^2 / 6 of the third derivative and by rounding,
    # 1e-5 of sums of some tens over 2 eps
    assert abs((up - down) / (2 * eps) - want) <= 0.02 * want + 1e-2


def _capture(fn):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        eager = [x.clone() for x in fn()]
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = list(fn())
    for x in out:
        x.fill_(float("nan"))  # the replay must write every output
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    pc.device_status()
    for a, b in zip(eager, out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_capture(dtype):
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, dy, w, b = r(300, 256).to(dtype), r(300, 256).to(dtype), r(256), r(256)
    _, mean, rstd = pc.layer_norm_fwd(x, w, b)
    _capture(lambda: pc.layer_norm_fwd(x, w, b))
    _capture(lambda: pc.layer_norm_bwd(dy, x, w, mean, rstd))
    q, k, v, do = (r(2, 700, 2, 64).to(dtype) for _ in range(4))
    decay, S = -torch.rand(2, generator=g, device="cuda"), r(2, 2, 64, 64)
    n = torch.tensor([700, 333], dtype=torch.int32, device="cuda")
    _capture(lambda: pc.linear_attention_fwd(q, k, v, decay, state=S, lengths=n))
    _capture(lambda: pc.linear_attention_bwd(q, k, v, decay, do, state=S, dstate=S.clone(), lengths=n).values())
    state = S.clone()

    def step():
        state.copy_(S)
        return [pc.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], decay, state), state]
    _capture(step)
    G = r(2, 200, 330).to(dtype)
    for precision in ("auto", "fp32"):
        _capture(lambda: [pc.orthogonalize(G, precision=precision)])
