"""The orthogonalised update of matrices that are small beside eps: X_0 = G / (|G|_F + eps) is then far
below one and grows by a step, and has to keep its bits at every size.

Tolerances, of the 2-norm of a matrix (see test_gpu_orthogonalize.py). While X is small a step
multiplies it by a, which carries relative errors over as they are; where it has grown, the polynomials
here have slopes below 1.6. Four roundings of 2.1e-4 a step (root mean square) then add up to
1.6 sqrt(4 steps) 2.1e-4; with operands of 22 bits, 2^-11 of that and the float32 sums', 5e-6 in five steps
and with the square root of their number in more."""
import numpy as np
import pytest
import torch

import log_space_sum_gb300 as pc
from oracle import factor_network as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pc.load()


def _of_norm(shape, norm, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    G = torch.randn(*shape, generator=gen, device="cuda")
    return G * (norm / G.norm(dim=(-1, -2), keepdim=True))


def _check(G, precision, steps, **kw):
    got = pc.orthogonalize(G, precision=precision, steps=steps, **kw).double().cpu().numpy()
    want = F.orthogonalize(G.double().cpu().numpy(), steps=steps, **kw)
    tol = 5e-6 * max(1.0, steps / 5) ** 0.5 if precision == "fp32" else 1.6 * (4 * steps) ** 0.5 * 2.1e-4
    err = np.sqrt(((got - want) ** 2).sum((-1, -2))) / np.sqrt((want ** 2).sum((-1, -2)))
    assert np.all(err <= tol), (err, tol)


@pytest.mark.parametrize("precision", ["auto", "fp32"])
@pytest.mark.parametrize("norm", [1e-7, 1e-10, 1e-12, 1e-14])
@pytest.mark.parametrize("shape", [(256, 512), (300, 96), (2, 131, 67)])
def test_small_beside_eps(shape, norm, precision):
    _check(_of_norm(shape, norm, 1), precision, 5)
    # far enough to reach one from any of these sizes, and part of the way
    for steps in (12, 60):
        _check(_of_norm(shape, norm, 2), precision, steps, coefficients=(2.0, -1.5, 0.5))


@pytest.mark.parametrize("precision", ["auto", "fp32"])
def test_matrices_of_different_size_and_a_large_eps(precision):
    G = torch.cat([_of_norm((1, 96, 160), n, i) for i, n in enumerate((1.0, 1e-9, 1e-13, 1e3))])
    _check(G, precision, 5)
    for i in range(4):  # none depends on its neighbours
        assert torch.equal(pc.orthogonalize(G, precision=precision)[i], pc.orthogonalize(G[i], precision=precision))
    _check(G[:1], precision, 5, eps=1e4)
    # a polynomial that lets X shrink
    _check(G, precision, 8, coefficients=(0.25, -0.1, 0.05))


def test_steps_on_the_gram_matrix():
    for norm in (1e-9, 1e-13):
        G = _of_norm((512, 46000), norm, 3)
        X = G.double()
        X = X / (X.norm() + 1e-7)
        for _ in range(7):
            A = X @ X.T
            X = 3.4445 * X + (-4.7750 * A + 2.0315 * (A @ A)) @ X
        got = pc.orthogonalize(G, steps=7).double()
        assert (got - X).norm() <= 2e-3 * X.norm()
