"""Host-side refusals of the factor network's entry points: the documented status before
anything is launched (no GPU)."""
import ctypes as C

import pytest
import torch

import log_space_sum_gb300 as pc
from log_space_sum_gb300 import _native as N
from log_space_sum_gb300 import build as B

FAKE = C.c_void_p(0x1000)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.load()


def _status(st):
    return N.STATUS[st]


def test_layer_norm(lib):
    f = lib.pc_layer_norm_fwd
    ok = [4, 8, FAKE, 8, None, None, 1e-5, FAKE, 8, None, None, 0, None]

    def call(**at):
        return _status(f(*[at.get(f"a{i}", x) for i, x in enumerate(ok)]))

    assert call(a11=2) == "PC_ERR_UNSUPPORTED"
    assert call(a0=-1) == "PC_ERR_SHAPE" and call(a1=0) == "PC_ERR_SHAPE" and call(a0=1 << 31) == "PC_ERR_SHAPE"
    assert call(a2=None) == "PC_ERR_NULL" and call(a7=None) == "PC_ERR_NULL"
    assert call(a3=7) == "PC_ERR_SHAPE" and call(a8=7) == "PC_ERR_SHAPE"
    assert call(a2=C.c_void_p(0x1002)) == "PC_ERR_ALIGNMENT"
    assert call(a6=-1.0) == "PC_ERR_SHAPE" and call(a6=float("nan")) == "PC_ERR_SHAPE"
    assert call(a0=0, a2=None) == "PC_OK"
    b = lib.pc_layer_norm_bwd
    args = [4, 8, FAKE, 8, FAKE, 8, None, FAKE, FAKE, FAKE, 8, FAKE, FAKE, 0, 0, FAKE, 1 << 30, None]

    def back(**at):
        return _status(b(*[at.get(f"a{i}", x) for i, x in enumerate(args)]))

    assert back(a7=None) == "PC_ERR_NULL" and back(a9=None) == "PC_ERR_NULL"
    assert back(a15=None) == "PC_ERR_WORKSPACE" and back(a16=4) == "PC_ERR_WORKSPACE"
    assert back(a15=C.c_void_p(0x1008)) == "PC_ERR_ALIGNMENT"
    nb = C.c_size_t(0)
    assert lib.pc_layer_norm_bwd_workspace(4, 8, C.byref(nb)) == 0 and nb.value >= 2 * 8 * 4


def test_linear_attention(lib):
    nb = C.c_size_t(0)
    query = lambda *a: _status(lib.pc_linear_attention_workspace(*a, C.byref(nb)))  # noqa: E731
    assert query(2, 8, 4, 64, 64, 1, 0) == "PC_OK"
    assert query(2, 8, 4, 64, 64, 1, 5) == "PC_ERR_UNSUPPORTED"
    assert query(2, 8, 0, 64, 64, 1, 0) == "PC_ERR_SHAPE" and query(-1, 8, 4, 64, 64, 1, 0) == "PC_ERR_SHAPE"
    assert query(2, 8, 4, 0, 64, 1, 0) == "PC_ERR_SHAPE" and query(2, 8, 4, 64, 257, 1, 0) == "PC_ERR_UNSUPPORTED"
    assert query(1 << 16, 8, 1 << 16, 64, 64, 1, 0) == "PC_ERR_SHAPE"
    st = (C.c_longlong * 21)(*([1] * 21))
    fwd = [2, 8, 4, 64, 64, FAKE, FAKE, FAKE, st, FAKE, 1.0, None, None, FAKE, None, 0, FAKE, 1 << 40, None]

    def call(**at):
        return _status(lib.pc_linear_attention_fwd(*[at.get(f"a{i}", x) for i, x in enumerate(fwd)]))

    for i in (5, 6, 7, 8, 9, 13):
        assert call(**{f"a{i}": None}) == "PC_ERR_NULL"
    assert call(a11=FAKE, a14=FAKE) == "PC_ERR_UNSUPPORTED"
    assert call(a6=C.c_void_p(0x1001)) == "PC_ERR_ALIGNMENT"
    assert call(a0=0) == "PC_OK"
    bwd = [2, 8, 4, 64, 64, FAKE, FAKE, FAKE, FAKE, st, FAKE, 1.0, None, None, None, FAKE, FAKE, FAKE, None, 0, FAKE,
           1 << 40, None]

    def back(**at):
        return _status(lib.pc_linear_attention_bwd(*[at.get(f"a{i}", x) for i, x in enumerate(bwd)]))

    for i in (5, 8, 9, 10, 15, 16, 17):
        assert back(**{f"a{i}": None}) == "PC_ERR_NULL"
    assert back(a13=FAKE, a18=FAKE) == "PC_ERR_UNSUPPORTED"
    step = [2, 4, 64, 64, FAKE, FAKE, FAKE, st, FAKE, 1.0, FAKE, FAKE, 0, None]
    for i in (4, 5, 6, 7, 8, 10, 11):
        assert _status(lib.pc_linear_attention_step(*[None if j == i else x for j, x in enumerate(step)])) == "PC_ERR_NULL"


def test_orthogonalize(lib):
    nb = C.c_size_t(0)
    query = lambda *a: _status(lib.pc_orthogonalize_workspace(*a, C.byref(nb)))  # noqa: E731
    assert query(1, 64, 32, 0) == "PC_OK" and nb.value > 0
    assert query(1, 64, 32, 7) == "PC_ERR_UNKNOWN_PRECISION"
    assert query(1, 0, 32, 0) == "PC_ERR_SHAPE" and query(1 << 16, 8, 8, 0) == "PC_ERR_SHAPE"
    ok = [1, 64, 32, FAKE, 5, 3.0, -4.0, 2.0, 1e-7, FAKE, 0, 0, FAKE, 1 << 40, None]

    def call(**at):
        return _status(lib.pc_orthogonalize(*[at.get(f"a{i}", x) for i, x in enumerate(ok)]))

    assert call(a3=None) == "PC_ERR_NULL" and call(a9=None) == "PC_ERR_NULL"
    assert call(a4=0) == "PC_ERR_SHAPE" and call(a8=-1.0) == "PC_ERR_SHAPE"
    assert call(a10=9) == "PC_ERR_UNSUPPORTED" and call(a11=9) == "PC_ERR_UNKNOWN_PRECISION"
    assert call(a12=None) == "PC_ERR_WORKSPACE" and call(a13=8) == "PC_ERR_WORKSPACE"
    assert call(a3=C.c_void_p(0x1004)) == "PC_ERR_ALIGNMENT"
    assert call(a0=0, a3=None) == "PC_OK"


def test_cpu_tensors_are_refused():
    x = torch.zeros(2, 8)
    for fn, args in ((pc.layer_norm_fwd, (x,)), (pc.layer_norm_bwd, (x, x, None, x[:, 0], x[:, 0])),
                     (pc.linear_attention_fwd, (x[None, None],) * 3 + (x[0],)),
                     (pc.linear_attention_step, (x[None],) * 3 + (x[0], x)), (pc.orthogonalize, (x,))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            fn(*args)
