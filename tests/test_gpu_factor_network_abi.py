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
