"""Device-side waits that run out in the factor network's tensor-core kernels: with a limit of 1 ns
the waits for products give up, the roles that this starves run into the default of 2 s, the timeout is
reported, nothing faults or hangs, and with the default limit back the same call gives the bits that
it gave before.

The cases (each with a product whose K loop outlasts a wait's first tries): products on clusters that share a tile (barriers whatever a wait decided) and on
persistent CTAs; attention in several segments, in order of time and against it, with tiles
that start before the sequence, whose weights eight warps exchange."""
import pytest
import torch

import log_space_sum_gb300 as pc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pc.load()
    pc.device_status()
    yield
    pc.set_wait_limit_ns(0)


def _runs_out_then_recovers(run):
    want = [t.clone() for t in run()]
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
    got = list(run())
    torch.cuda.synchronize()
    pc.device_status()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("shape,steps", [((300, 40000), 5), ((8, 2048, 2048), 1), ((1024, 16384), 5)])
def test_orthogonalize(shape, steps):
    gen = torch.Generator(device="cuda").manual_seed(1)
    G = torch.randn(*shape, generator=gen, device="cuda")
    _runs_out_then_recovers(lambda: [pc.orthogonalize(G, steps=steps)])


@pytest.mark.parametrize("B,T,H,dk,dv", [(1, 3000, 2, 128, 128), (2, 1500, 3, 128, 72)])
def test_linear_attention(B, T, H, dk, dv):
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k = (r(B, T, H, dk).bfloat16() for _ in range(2))
    v, do = (r(B, T, H, dv).bfloat16() for _ in range(2))
    decay, S, dS = -0.1 * torch.rand(H, generator=gen, device="cuda"), r(B, H, dk, dv), r(B, H, dk, dv)
    n = torch.randint(T // 2, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    _runs_out_then_recovers(lambda: pc.linear_attention_fwd(q, k, v, decay, state=S, lengths=n))
    _runs_out_then_recovers(lambda: pc.linear_attention_bwd(q, k, v, decay, do, state=S, dstate=dS, lengths=n).values())
