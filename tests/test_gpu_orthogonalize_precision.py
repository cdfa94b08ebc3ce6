"""Precision "fp32" of the orthogonalised update on small float32 matrices of a few strong directions
over a full-rank floor, as gradients are.

Tolerance, of the 2-norm. Operands of 22 bits: 7e-7 in five steps (2^-11 of the 1.5e-3 of 11 bits, see
test_gpu_orthogonalize.py). The accumulator truncates: each of the twelve products that a block of 64
adds to it costs up to 2^-24, 7e-7 of a value for a slice of one block, three products a step, slope 1.6:
half of it on average, so 1.6 sqrt(15) 3.6e-7 = 2.2e-6. Together 2.9e-6."""
import math

import pytest
import torch

import log_space_sum_gb300 as pc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(6, 770, 333), (1, 100, 100), (4, 300, 1000), (1, 64, 900), (1, 400, 90), (2, 150, 700)])
def test_small_gradients(shape):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    batch, m, n = shape
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    rank = max(1, min(m, n) // 16)
    G = (r(batch, m, n) + r(batch, m, rank) @ r(batch, rank, n) / math.sqrt(rank) * 2) * 1e-3
    X = G.double().mT if m > n else G.double()
    X = X / (X.norm(dim=(-1, -2), keepdim=True) + 1e-7)
    for _ in range(5):
        A = X @ X.mT
        X = 3.4445 * X + (-4.7750 * A + 2.0315 * (A @ A)) @ X
    want = X.mT if m > n else X
    got = pc.orthogonalize(G, precision="fp32").double()
    assert ((got - want).norm(dim=(-1, -2)) <= 2.9e-6 * want.norm(dim=(-1, -2))).all()
