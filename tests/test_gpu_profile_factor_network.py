"""What pc_profile_start / _stop record of the factor network's operators: every contraction, with its
algorithmic flops (each product once)."""
import pytest
import torch

import log_space_sum_gb300 as pc

pytestmark = pytest.mark.gpu


def _record(fn):
    fn()
    torch.cuda.synchronize()
    pc.profile_start(64)
    try:
        fn()
    finally:
        got = pc.profile_stop(64)
    return got


@pytest.mark.parametrize("dtype,B,T,H,dk,dv", [(torch.bfloat16, 2, 300, 3, 128, 64), (torch.bfloat16, 1, 4000, 2, 128, 128),
                                               (torch.bfloat16, 400, 60, 2, 64, 64), (torch.float32, 2, 200, 3, 40, 56)])
def test_linear_attention(dtype, B, T, H, dk, dv):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    q, k, v, do = r(B, T, H, dk), r(B, T, H, dk), r(B, T, H, dv), r(B, T, H, dv)
    decay = -torch.rand(H, generator=gen, device="cuda")
    for flops, fn in ((4, lambda: pc.linear_attention_fwd(q, k, v, decay)),
                      (10, lambda: pc.linear_attention_bwd(q, k, v, decay, do))):
        [(kind, ms, got, launches)] = _record(fn)
        assert kind == "linear_attention" and got == flops * B * T * H * dk * dv
        assert 1 <= launches <= 4 and 0 < ms < 1000


def test_orthogonalize_and_what_is_no_contraction():
    G = torch.randn(100, 200, device="cuda")
    got = _record(lambda: pc.orthogonalize(G, steps=2))
    assert [kind for kind, *_ in got] == ["orthogonalize"] * 6
    assert sum(flops for _, _, flops, _ in got) == 2 * (3 * 100 * 100 * 200 + 100 ** 3)
    assert _record(lambda: pc.layer_norm_fwd(G)) == []
