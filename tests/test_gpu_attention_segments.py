"""Segmented attention without a pause between calls: the launch that leaves the segments' states
starts while the last call's pass ends, and its own pass beside it. No wait runs out, equal bits."""
import pytest
import torch

import log_space_sum_gb300 as pc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,H,dk,dv", [(4, 2000, 16, 128, 128), (1, 9000, 5, 64, 128), (3, 1100, 4, 128, 64),
                                         (2, 1500, 8, 64, 64)])
def test_back_to_back(B, T, H, dk, dv):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    decay, cases = -0.1 * torch.rand(H, generator=gen, device="cuda"), []
    for i in range(3):
        q, k = (r(B, T, H, dk).bfloat16() for _ in range(2))
        v, do = (r(B, T, H, dv).bfloat16() for _ in range(2))
        n = torch.randint(T // 2, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        cases.append(dict(q=q, k=k, v=v, log_decay=decay, state=r(B, H, dk, dv), lengths=n if i else None))
        cases[-1]["do"] = do

    def run(case, way):
        kw = dict(case)
        if way == "bwd":
            return list(pc.linear_attention_bwd(dstate=kw["state"], **kw).values())
        kw.pop("do")
        return list(pc.linear_attention_fwd(**kw))

    pc.device_status()
    for way, calls in (("fwd", 600), ("bwd", 150)):
        want = [[t.clone() for t in run(c, way)] for c in cases]
        torch.cuda.synchronize()
        same = []
        for i in range(calls):
            got = run(cases[i % 3], way)
            if i % 7 == 0:
                same.append(torch.stack([(a == b).all() for a, b in zip(got, want[i % 3])]).all())
        pc.device_status()
        assert torch.stack(same).all()
