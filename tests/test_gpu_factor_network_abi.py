"""The factor network's operators through the C ABI, at the edges of what the header promises
(a workspace that is aligned to 16 bytes and no more)."""
import ctypes as C

import pytest
import torch

import log_space_sum_gb300 as pc
from log_space_sum_gb300 import _native as N

pytestmark = pytest.mark.gpu
CODE = {torch.float32: 0, torch.bfloat16: 1}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pc.load()


def _stream():
    return torch.cuda.current_stream().cuda_stream


class _Workspace:
    """`bytes` bytes that start `shift` bytes past a 512-byte boundary, between guards."""

    GUARD = 4096

    def __init__(self, nbytes, shift):
        self.all = torch.full((2 * self.GUARD + shift + nbytes,), 0xA5, dtype=torch.uint8, device="cuda")
        assert self.all.data_ptr() % 512 == 0
        self.first, self.bytes = self.GUARD + shift, nbytes
        self.ptr = self.all.data_ptr() + self.first

    def untouched_around(self):
        return bool((self.all[:self.first] == 0xA5).all() and (self.all[self.first + self.bytes:] == 0xA5).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape,precision", [((2, 130, 70), "auto"), ((2, 130, 70), "fp32"), ((1, 333, 770), "tf32"),
                                             ((1, 512, 46000), "auto")])
def test_orthogonalize_workspace_aligned_to_16_bytes(shape, precision, dtype):
    """The operands are read 32 bytes at a time wherever the workspace starts: the same bits."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    G = torch.randn(*shape, generator=gen, device="cuda").to(dtype)
    want = pc.orthogonalize(G, precision=precision)
    prec, need = pc.precision_code(precision), C.c_size_t(0)
    N.call("pc_orthogonalize_workspace", *shape, prec, C.byref(need))
    for shift in (0, 16, 32, 48, 240):
        ws, out = _Workspace(need.value, shift), torch.zeros_like(G)
        N.call("pc_orthogonalize", *shape, G.data_ptr(), 5, 3.4445, -4.7750, 2.0315, 1e-7, out.data_ptr(), CODE[dtype],
               prec, ws.ptr, ws.bytes, _stream())
        pc.device_status()
        assert torch.equal(out, want), shift
        assert ws.untouched_around(), shift


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,dim,first", [(700, 1024, 0), (900, 513, 3), (60, 4097, 1), (30, 9000, 0)])
def test_layer_norm_gradient_in_the_place_of_its_inputs(rows, dim, first, dtype):
    """dx over dy and over x: the bits of a dx of its own at the same place in a 16-byte piece (at
    another, the rows are taken value by value and summed in another order)."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    place = lambda: r(rows * dim + 8).to(dtype)[first:first + rows * dim].view(rows, dim)  # noqa: E731
    x, dy, w = place(), place(), r(dim)
    _, mean, rstd = pc.layer_norm_fwd(x, w)
    want = pc.layer_norm_bwd(dy, x, w, mean, rstd, dx=place())
    for over in (0, 1):
        a, b = place().copy_(x), place().copy_(dy)
        got = pc.layer_norm_bwd(b, a, w, mean, rstd, dx=(b, a)[over])
        assert all(torch.equal(p, q) for p, q in zip(got, want))
