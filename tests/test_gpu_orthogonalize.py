"""GPU parity of the orthogonalised update (pc_orthogonalize) against the float64 products
and against the polynomial on the singular values.

Tolerances, of the 2-norm of a matrix. An operand of 11 significant bits is off by 2^-11 at
most, 2.1e-4 in the root mean square; a step rounds X twice and A and B once, and over five
steps with the polynomial's slope (below 1.6 on singular values that have grown; small ones
grow by their slope, so that their relative errors carry over) these add up to at most
sqrt(20) 2.1e-4 1.6 = 1.5e-3, and 2e-3 is allowed. With few rows one rounding of A or B bears
on a large part of X, and the greatest error takes the place of the root mean square:
sqrt(20) 2^-11 1.6 = 3.5e-3. Operands of 22 bits: 2^-11 of that and the float32 sums'
2^-24 sqrt(N) a product, 5e-6. bf16 outputs add 1.7e-3 (root mean square; 2^-8 at most).
Where a few directions hold the matrix, rounding fills the others with noise of an operand's
relative error, which grows like any small singular value by at most 3.4445 a step, 485 in
all, whatever the arithmetic: 485 times twice 2.1e-4, or twice 1e-7 (22 bits), absolute, as
|X_0|_F = 1."""
import numpy as np
import pytest
import torch

import log_space_sum_gb300 as pc
from oracle import factor_network as F

pytestmark = pytest.mark.gpu
REL = {"auto": 2e-3, "tf32": 2e-3, "fp32": 5e-6}
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pc.load()


def _draw(shape, dtype, seed, size=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (size * torch.randn(*shape, generator=g, device="cuda")).to(TYPES[dtype])


def _check(G, precision, noise=0.0, **kw):
    X = pc.orthogonalize(G, precision=precision, **kw)
    want = F.orthogonalize(G.double().cpu().numpy(), **kw)
    X = X.double().cpu().numpy()
    few = min(G.shape[-2:]) < 16
    tol = max(REL[precision], 3.5e-3 if few and precision != "fp32" else 0)
    tol += (2.0 ** -8 if few else 1.7e-3) if G.dtype == torch.bfloat16 else 0
    assert X.shape == want.shape
    err = np.sqrt(((X - want) ** 2).sum((-1, -2)))
    assert np.all(err <= tol * np.sqrt((want ** 2).sum((-1, -2))) + noise), err
    return X


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("precision", ["auto", "tf32", "fp32"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 40), (37, 1), (5, 7), (64, 64), (128, 200), (200, 128), (129, 257),
                                   (3, 96, 160), (2, 2, 130, 66), (333, 770), (512, 512)])
def test_sizes(shape, precision, dtype):
    _check(_draw(shape, dtype, sum(shape)), precision)


@pytest.mark.parametrize("precision", ["auto", "fp32"])
def test_larger(precision):
    _check(_draw((700, 2100), "fp32", 1), precision)


@pytest.mark.parametrize("precision", ["auto", "fp32"])
@pytest.mark.parametrize("size", [1e-12, 1.0, 1e12])
def test_scale_of_the_input_does_not_matter(precision, size):
    _check(_draw((96, 160), "fp32", 2, size), precision, eps=0.0)


def test_singular_values():
    """A spectrum over three decades: each singular value goes where the polynomial sends it."""
    rng = np.random.default_rng(3)
    U, _ = np.linalg.qr(rng.normal(size=(160, 160)))
    V, _ = np.linalg.qr(rng.normal(size=(300, 160)))
    s = np.logspace(0, -3, 160)
    X = pc.orthogonalize(torch.tensor(U * s @ V.T, dtype=torch.float32, device="cuda"), precision="fp32")
    p = s / np.linalg.norm(s)
    for _ in range(5):
        p = 3.4445 * p - 4.7750 * p ** 3 + 2.0315 * p ** 5
    got = np.diag(U.T @ X.double().cpu().numpy() @ V)
    np.testing.assert_allclose(got, p, atol=2e-5)


@pytest.mark.parametrize("precision", ["auto", "fp32"])
def test_rank_one_and_uneven_matrices(precision):
    g = _draw((150, 90), "fp32", 4, 1.0)
    noise = 2 * 485 * (1e-7 if precision == "fp32" else 2.1e-4)
    X = _check(torch.outer(g[:, 0], g[0]), precision, noise)
    u, v = (t.double().cpu().numpy() / t.double().norm().item() for t in (g[:, 0], g[0]))
    p = 1.0
    for _ in range(5):
        p = 3.4445 * p - 4.7750 * p ** 3 + 2.0315 * p ** 5
    assert abs(u @ X @ v - p) <= 3.5e-3 * p  # the direction itself
    g[:, 3] *= 1e4  # one column holds nearly all of the norm
    _check(g, precision, noise)
    spike = torch.zeros(64, 200, device="cuda")
    spike[5, 7] = 2.0
    assert np.count_nonzero(_check(spike, precision, noise)) == 1


def test_zeros_and_non_finite_stay_in_their_matrix():
    g = _draw((4, 70, 50), "fp32", 5)
    g[1] = 0
    g[2, 3, 4] = float("nan")
    X = pc.orthogonalize(g)
    assert not X[1].any() and torch.isnan(X[2]).all()
    for i in (0, 3):
        assert torch.equal(X[i], pc.orthogonalize(g[i]))


def test_steps_coefficients_in_place_and_streams():
    g = _draw((2, 100, 60), "fp32", 6)
    X = _check(g, "fp32", steps=1)
    _check(g, "fp32", steps=12, coefficients=(2.0, -1.5, 0.5))  # converges: X^T X = 1
    Y = pc.orthogonalize(g, steps=40, coefficients=(2.0, -1.5, 0.5), precision="fp32").double()
    np.testing.assert_allclose((Y.transpose(1, 2) @ Y).cpu().numpy(), np.eye(60)[None].repeat(2, 0), atol=2e-5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        own = g.clone()
        pc.orthogonalize(own, steps=1, precision="fp32", out=own)
    torch.cuda.current_stream().wait_stream(side)
    np.testing.assert_array_equal(own.double().cpu().numpy(), X)
    assert pc.orthogonalize(torch.empty(0, 8, 8, device="cuda")).shape == (0, 8, 8)


def test_refusals():
    g = _draw((8, 8), "fp32", 7)
    with pytest.raises(TypeError, match="G must be torch.float32 or"):
        pc.orthogonalize(g.double())
    with pytest.raises(ValueError, match="at least two"):
        pc.orthogonalize(g[0])
    with pytest.raises(ValueError, match="contiguous"):
        pc.orthogonalize(g.t()[:, :4])
    with pytest.raises(ValueError, match="unknown precision"):
        pc.orthogonalize(g, precision="fp16")
    with pytest.raises(pc.PCError, match="steps"):
        pc.orthogonalize(g, steps=0)
    with pytest.raises(pc.PCError, match="PC_ERR_ALIGNMENT"):
        pc.orthogonalize(_draw((65,), "fp32", 8)[1:].view(8, 8))


def _exact(G, coefficients=(3.4445, -4.7750, 2.0315), steps=5):
    """The formula in float64 on the device (the matrices are large)."""
    a, b, c = coefficients
    X = G.double().mT if G.shape[-2] > G.shape[-1] else G.double()
    X = X / (X.norm(dim=(-1, -2), keepdim=True) + 1e-7)
    for _ in range(steps):
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.mT if G.shape[-2] > G.shape[-1] else X


@pytest.mark.parametrize("shape", [(1024, 16384), (16500, 1000), (3, 520, 16001)])
def test_very_wide(shape):
    """Steps on the Gram matrix in two parts. A G of 8 bits is exact in float16, so what is left
    is 2^-22 an operand and the accumulator's truncation, at most 2^-24 for each of the N / 16
    additions, 6e-5 of A (3e-5 of X); with the slope of five steps on singular values that are
    all alike (their errors carry over as they are): 2e-4 allowed."""
    G = _draw(shape, "bf16", 11)
    want = _exact(G)
    norm = want.norm(dim=(-1, -2))
    X = pc.orthogonalize(G.float())
    assert ((X.double() - want).norm(dim=(-1, -2)) <= 2e-4 * norm).all()
    X = pc.orthogonalize(G)
    assert X.dtype == torch.bfloat16
    assert ((X.double() - want).norm(dim=(-1, -2)) <= (2e-4 + 1.7e-3) * norm).all()
    G = _draw(shape, "fp32", 12)  # rounded to 11 bits
    want = _exact(G)
    assert ((pc.orthogonalize(G).double() - want).norm(dim=(-1, -2)) <= 2e-3 * norm).all()


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 7, 11])
def test_very_wide_steps(steps):
    """One step, several on one Gram matrix, and more than one of those; X is rounded in between."""
    G = _draw((512, 46000), "bf16", 13).float()
    want = _exact(G, steps=steps)
    X = pc.orthogonalize(G, steps=steps)
    assert (X.double() - want).norm() <= 2e-3 * want.norm()
    coefficients = (1.5, -0.5, 0.0)
    want = _exact(G, coefficients, steps)
    X = pc.orthogonalize(G, steps=steps, coefficients=coefficients)
    assert (X.double() - want).norm() <= 2e-3 * want.norm()


def test_very_wide_uneven():
    """Directions of very different size: the noise of two-part operands, 485 times 2e-7 of the
    matrix, and 2e4 times 2e-7 of A's in the slope of B's share, absolute."""
    g = _draw((512, 46000), "bf16", 14, 1.0).float()
    one = torch.outer(g[:, 0], g[0]).bfloat16().float()
    for G in (one, one + 1e-3 * g.sign(), torch.cat([1e3 * g[:1], g[1:]])):
        G = G.bfloat16().float()
        want = _exact(G)
        assert (pc.orthogonalize(G).double() - want).norm() <= 2e-3 * want.norm() + 485 * 2e-7 + 2e4 * 2e-7 * 4.775
    G = g.clone()
    G[3, 5] = float("inf")
    assert not torch.isfinite(pc.orthogonalize(G)).any()
    assert not pc.orthogonalize(torch.zeros_like(g)).any()
