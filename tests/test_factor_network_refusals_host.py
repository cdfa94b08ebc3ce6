"""Refusals of the factor network's entry points beyond their types and shapes: before anything is
launched (no GPU)."""
import ctypes as C

import pytest

from log_space_sum_gb300 import _native as N
from log_space_sum_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.load()


def _places(n):
    """n pointers, all different and 16-byte aligned."""
    return [C.c_void_p(0x10000 * (i + 1)) for i in range(n)]


def _strides(tensors, H=4, D=64, T=8):
    return (C.c_longlong * (3 * tensors))(*([T * H * D, H * D, D] * tensors))


def _forward(lib, q, k, v, o, state=None, state_out=None, strides=None):
    return N.STATUS[lib.pc_linear_attention_fwd(2, 8, 4, 64, 64, q, k, v, strides or _strides(4), C.c_void_p(0x8000), 1.0,
                                                state, None, o, state_out, 0, C.c_void_p(0x4000), 0, None)]


def _backward(lib, tensors, state=None, dstate_out=None, dstate=None, strides=None):
    q, k, v, do, dq, dk, dv = tensors
    return N.STATUS[lib.pc_linear_attention_bwd(2, 8, 4, 64, 64, q, k, v, do, strides or _strides(7), C.c_void_p(0x8000),
                                                1.0, state, dstate_out, None, dq, dk, dv, dstate, 0,
                                                C.c_void_p(0x4000), 0, None)]


def test_attention_outputs_that_are_inputs(lib):
    q, k, v, o, s = _places(5)
    for same in (q, k, v):
        assert _forward(lib, q, k, v, same) == "PC_ERR_UNSUPPORTED"
        assert b"o may not be" in lib.pc_last_error()
    assert _forward(lib, q, k, v, o, s, s) == "PC_ERR_UNSUPPORTED"


def test_attention_gradients_that_are_inputs_or_one_another(lib):
    t = _places(7)
    for i in range(4, 7):
        for j in range(i):
            same = list(t)
            same[i] = t[j]
            assert _backward(lib, same) == "PC_ERR_UNSUPPORTED", (i, j)
            assert b"may not be" in lib.pc_last_error()


def test_attention_state_gradient_in_the_state(lib):
    t, (s, ds) = _places(7), (C.c_void_p(0x900000), C.c_void_p(0x980000))
    assert _backward(lib, t, state=s, dstate_out=ds, dstate=s) == "PC_ERR_UNSUPPORTED"
    assert b"dstate may not be state" in lib.pc_last_error()
    assert _backward(lib, t, state=s, dstate_out=ds, dstate=ds) == "PC_ERR_UNSUPPORTED"


def test_attention_outputs_whose_elements_share_memory(lib):
    """An input may be shared by heads or sequences (stride 0); an output would be written by several
    parts at once."""
    q, k, v, o = _places(4)
    for dim in range(3):
        st = _strides(4)
        st[9 + dim] = 0
        assert _forward(lib, q, k, v, o, strides=st) == "PC_ERR_SHAPE"
        assert b"o: stride 0" in lib.pc_last_error()
        for tensor in range(4, 7):
            st = _strides(7)
            st[3 * tensor + dim] = 0
            assert _backward(lib, _places(7), strides=st) == "PC_ERR_SHAPE"
            assert b"stride 0" in lib.pc_last_error()
    for dim in range(2):
        st = (C.c_longlong * 8)(*([256, 64] * 4))
        st[6 + dim] = 0
        got = lib.pc_linear_attention_step(2, 4, 64, 64, q, k, v, st, C.c_void_p(0x8000), 1.0, C.c_void_p(0x9000), o, 0, None)
        assert N.STATUS[got] == "PC_ERR_SHAPE"


def test_attention_workspace_with_backward_serves_both_directions(lib):
    """The gradient's passes are three times the heads and may be cut into fewer segments."""
    def size(shape, back, dtype):
        nb = C.c_size_t(0)
        assert lib.pc_linear_attention_workspace(*shape, back, dtype, C.byref(nb)) == 0
        return nb.value

    for dtype in (0, 1):
        for shape in [(1, 1500, 5, 128, 128)] + [(B, T, H, dk, dv) for B in (1, 2, 4) for T in (33, 333, 1500, 4000, 20000)
                                                 for H in (1, 3, 5, 16) for dk, dv in ((64, 64), (128, 64), (40, 56))]:
            assert size(shape, 1, dtype) >= size(shape, 0, dtype), (shape, dtype)


def test_attention_gradient_of_too_many_heads(lib):
    """A gradient on the tensor cores launches a column of CTAs for each head of each of three passes."""
    t = _places(7)
    st = _strides(7, H=1 << 15, D=8, T=1)
    got = lib.pc_linear_attention_bwd(1 << 15, 1, 1 << 15, 8, 8, *t[:4], st, C.c_void_p(0x8000), 1.0, None, None, None, *t[4:],
                                      None, 1, None, 0, None)
    assert N.STATUS[got] == "PC_ERR_SHAPE" and b"fewer than 2^31" in lib.pc_last_error()


def test_layer_norm_in_place_at_another_stride(lib):
    x, dy, m, s, ws = _places(5)
    fwd = lambda y, ld, rows=4: N.STATUS[lib.pc_layer_norm_fwd(rows, 8, x, 16, None, None, 1e-5, y, ld, None, None, 0, None)]  # noqa: E731
    assert fwd(x, 8) == "PC_ERR_SHAPE" and b"another row stride" in lib.pc_last_error()

    def bwd(dx, ld):
        return N.STATUS[lib.pc_layer_norm_bwd(4, 8, dy, 8, x, 16, None, m, s, dx, ld, None, None, 0, 0, ws, 1 << 20, None)]

    assert bwd(dy, 16) == "PC_ERR_SHAPE" and b"another row stride" in lib.pc_last_error()
    assert bwd(x, 8) == "PC_ERR_SHAPE" and b"another row stride" in lib.pc_last_error()
