"""Host-side refusals of softmax attention, the norms with rotation and the paged cache: the documented
status before anything is launched (no GPU)."""
import ctypes as C
import math

import pytest
import torch

import log_space_sum_gb300 as pc
from log_space_sum_gb300 import _native as N
from log_space_sum_gb300 import build as B

P = [C.c_void_p(0x10000 * (i + 1)) for i in range(16)]  # places, all different
ODD = C.c_void_p(0x10001)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.load()


def _caller(f, args):
    return lambda **at: N.STATUS[f(*[at.get(f"a{i}", x) for i, x in enumerate(args)])]


def _ll(*v):
    return (C.c_longlong * len(v))(*v)


def _replace(values, i, x):
    v = list(values)
    v[i] = x
    return _ll(*v)


def test_qk_norm_rotary_fwd(lib):
    st = [512, 64, 128, 64, 512, 64, 128, 64]
    call = _caller(lib.pc_qk_norm_rotary_fwd, [4, 8, 2, 64, 32, P[0], P[1], _ll(*st), None, None, P[2], P[3], 1e-6, 1.0, 0, 1,
                                               P[4], P[5], 0, None])
    assert call(a18=2) == "PC_ERR_UNSUPPORTED" and call(a14=2) == "PC_ERR_UNSUPPORTED"
    assert call(a3=257) == "PC_ERR_UNSUPPORTED" and call(a3=0) == "PC_ERR_SHAPE"
    for bad in (-2, 3, 66):
        assert call(a4=bad) == "PC_ERR_SHAPE"
    assert call(a0=-1) == "PC_ERR_SHAPE" and call(a0=1 << 31) == "PC_ERR_SHAPE"
    assert call(a1=0, a2=0) == "PC_ERR_SHAPE" and call(a1=-1) == "PC_ERR_SHAPE" and call(a2=65536) == "PC_ERR_SHAPE"
    for i in (5, 6, 7, 10, 11, 16, 17):
        assert call(**{f"a{i}": None}) == "PC_ERR_NULL", i
    assert call(a5=ODD) == "PC_ERR_ALIGNMENT" and call(a17=ODD) == "PC_ERR_ALIGNMENT"
    for bad in (-1.0, float("nan"), float("inf")):
        assert call(a12=bad) == "PC_ERR_SHAPE"
    assert call(a13=float("nan")) == "PC_ERR_SHAPE"
    assert call(a16=P[0], a7=_replace(st, 4, 1024)) == "PC_ERR_SHAPE" and b"other strides" in lib.pc_last_error()
    assert call(a17=P[4]) == "PC_ERR_UNSUPPORTED"
    assert call(a17=P[0]) == "PC_ERR_UNSUPPORTED" and call(a16=P[1]) == "PC_ERR_UNSUPPORTED"
    for i in range(4, 8):
        assert call(a7=_replace(st, i, 0)) == "PC_ERR_SHAPE" and b"stride 0" in lib.pc_last_error()
    assert call(a0=0, a5=None) == "PC_OK"


def test_qk_norm_rotary_bwd(lib):
    nb = C.c_size_t(0)
    assert lib.pc_qk_norm_rotary_bwd_workspace(4, 8, 2, 64, 1, C.byref(nb)) == 0 and nb.value >= 2 * 64 * 4
    need = nb.value
    assert lib.pc_qk_norm_rotary_bwd_workspace(4, 8, 2, 64, 0, C.byref(nb)) == 0 and nb.value == 0
    assert N.STATUS[lib.pc_qk_norm_rotary_bwd_workspace(4, 8, 2, 64, 1, None)] == "PC_ERR_NULL"
    st = [512, 64, 128, 64] * 3
    call = _caller(lib.pc_qk_norm_rotary_bwd, [4, 8, 2, 64, 32, P[0], P[1], P[2], P[3], _ll(*st), None, None, P[4], P[5], 1e-6,
                                               1.0, 0, 1, P[6], P[7], P[8], P[9], 0, 0, P[10], need, None])
    for i in (5, 6, 7, 8, 9, 12, 13, 18, 19):
        assert call(**{f"a{i}": None}) == "PC_ERR_NULL", i
    assert call(a24=None) == "PC_ERR_WORKSPACE" and call(a25=need - 1) == "PC_ERR_WORKSPACE"
    assert call(a24=C.c_void_p(0x10008)) == "PC_ERR_ALIGNMENT"
    assert call(a18=P[2], a9=_replace(st, 8, 1024)) == "PC_ERR_SHAPE"
    assert call(a18=P[0], a9=_replace(st, 9, 128)) == "PC_ERR_SHAPE"
    assert call(a19=P[6]) == "PC_ERR_UNSUPPORTED"
    for i in (18, 19):
        for j in ((1, 3) if i == 18 else (0, 2)):
            assert call(**{f"a{i}": P[j]}) == "PC_ERR_UNSUPPORTED", (i, j)


def test_attention_fwd(lib):
    st = [512, 64, 128, 64, 128, 64, 512, 64]
    call = _caller(lib.pc_attention_fwd, [2, 10, 8, 2, 64, P[0], P[1], P[2], _ll(*st), P[3], 0.1, P[4], P[5], 0, None])
    assert call(a13=2) == "PC_ERR_UNSUPPORTED" and call(a4=257) == "PC_ERR_UNSUPPORTED"
    assert call(a4=0) == "PC_ERR_SHAPE" and call(a3=3) == "PC_ERR_SHAPE" and call(a3=0) == "PC_ERR_SHAPE"
    assert call(a0=-1) == "PC_ERR_SHAPE" and call(a1=-1) == "PC_ERR_SHAPE" and call(a1=1 << 30) == "PC_ERR_SHAPE"
    assert call(a2=65536, a3=1) == "PC_ERR_SHAPE"
    for i in (5, 6, 7, 8, 11):
        assert call(**{f"a{i}": None}) == "PC_ERR_NULL", i
    for i in (5, 6, 7, 11):
        assert call(**{f"a{i}": ODD}) == "PC_ERR_ALIGNMENT", i
    for i in range(3):
        assert call(a11=P[i]) == "PC_ERR_UNSUPPORTED"
    for i in (6, 7):
        assert call(a8=_replace(st, i, 0)) == "PC_ERR_SHAPE"
    assert call(a9=None, a1=9) == "PC_ERR_SHAPE" and b"multiple of B" in lib.pc_last_error()
    assert call(a0=0, a5=None) == "PC_OK" and call(a1=0, a5=None) == "PC_OK"


def test_attention_bwd(lib):
    nb = C.c_size_t(0)
    assert lib.pc_attention_bwd_workspace(2, 10, 8, 2, 64, 1, C.byref(nb)) == 0 and nb.value >= 10 * 8 * 4
    need = nb.value
    assert N.STATUS[lib.pc_attention_bwd_workspace(2, 10, 8, 3, 64, 1, C.byref(nb))] == "PC_ERR_SHAPE"
    st = [512, 64, 128, 64, 128, 64, 512, 64, 512, 64, 512, 64, 128, 64, 128, 64]
    args = [2, 10, 8, 2, 64, P[0], P[1], P[2], P[3], P[4], _ll(*st), P[5], 0.1, P[6], P[7], P[8], P[9], 1, P[10], need, None]
    call = _caller(lib.pc_attention_bwd, args)
    for i in (5, 6, 7, 8, 9, 10, 13, 14, 15, 16):
        assert call(**{f"a{i}": None}) == "PC_ERR_NULL", i
    assert call(a18=None) == "PC_ERR_WORKSPACE" and call(a19=need - 1) == "PC_ERR_WORKSPACE"
    assert call(a18=C.c_void_p(0x10008)) == "PC_ERR_ALIGNMENT"
    for i in range(14, 17):
        for j in list(range(5, 10)) + list(range(14, i)):
            assert call(**{f"a{i}": args[j]}) == "PC_ERR_UNSUPPORTED", (i, j)
    for i in range(10, 16):
        assert call(a10=_replace(st, i, 0)) == "PC_ERR_SHAPE", i


def test_paged_attention(lib):
    nb = C.c_size_t(0)
    size = lambda *a: N.STATUS[lib.pc_paged_attention_workspace(*a, C.byref(nb))]  # noqa: E731
    assert size(2, 10, 8, 2, 64, 7, 16, 4, 1) == "PC_OK"
    need = nb.value
    assert size(2, 10, 8, 2, 64, -1, 16, 4, 1) == "PC_ERR_SHAPE" and size(2, 10, 8, 2, 64, 7, 0, 4, 1) == "PC_ERR_SHAPE"
    assert size(2, 10, 8, 2, 64, 7, 1 << 20, 1 << 20, 1) == "PC_ERR_SHAPE" and size(2, 10, 8, 2, 64, 7, 16, 4, 3) == "PC_ERR_UNSUPPORTED"
    st = [512, 64, 2048, 128, 64, 2048, 128, 64, 512, 64]
    call = _caller(lib.pc_paged_attention, [2, 10, 8, 2, 64, 7, 16, 4, P[0], P[1], P[2], _ll(*st), P[3], P[4], P[5], 0.1, P[6],
                                            None, 1, P[7], need, None])
    for i in (8, 9, 10, 11, 12, 13, 16):
        assert call(**{f"a{i}": None}) == "PC_ERR_NULL", i
    for i in (8, 9, 10, 16):
        assert call(**{f"a{i}": ODD}) == "PC_ERR_ALIGNMENT", i
    for i in range(3):
        assert call(a16=P[i]) == "PC_ERR_UNSUPPORTED"
    assert call(a14=None, a1=9) == "PC_ERR_SHAPE"
    for i in (8, 9):
        assert call(a11=_replace(st, i, 0)) == "PC_ERR_SHAPE"
    assert call(a0=0, a8=None) == "PC_OK"
    # ranges of a long cache need a workspace
    assert size(1, 1, 8, 2, 64, 7000, 16, 4096, 0) == "PC_OK" and nb.value > 0
    long = [1, 1, 8, 2, 64, 7000, 16, 4096, P[0], P[1], P[2], _ll(*st), P[3], P[4], P[5], 0.1, P[6], None, 0, P[7], nb.value, None]
    call = _caller(lib.pc_paged_attention, long)
    assert call(a19=None) == "PC_ERR_WORKSPACE" and call(a20=nb.value - 1) == "PC_ERR_WORKSPACE"
    assert call(a19=C.c_void_p(0x10008)) == "PC_ERR_ALIGNMENT"


def test_paged_plan_and_write(lib):
    call = _caller(lib.pc_paged_plan, [2, 4, 16, 5, 10, P[0], P[1], P[2], P[3], P[4], P[5], P[6], P[7], P[8], None])
    for i in range(5, 14):
        assert call(**{f"a{i}": None}) == "PC_ERR_NULL", i
    for i in (0, 1, 3, 4):
        assert call(**{f"a{i}": -1}) == "PC_ERR_SHAPE", i
    assert call(a2=0) == "PC_ERR_SHAPE" and call(a0=16385) == "PC_ERR_UNSUPPORTED"
    for i in range(8, 14):
        assert call(**{f"a{i}": P[0]}) == "PC_ERR_UNSUPPORTED", i
    st = [128, 64, 128, 64, 2048, 128, 64, 2048, 128, 64]
    call = _caller(lib.pc_paged_write, [10, 2, 64, 7, 16, P[0], P[1], _ll(*st), P[2], P[3], P[4], 1, None])
    for i in (5, 6, 7, 8, 9, 10):
        assert call(**{f"a{i}": None}) == "PC_ERR_NULL", i
    assert call(a11=7) == "PC_ERR_UNSUPPORTED" and call(a0=-1) == "PC_ERR_SHAPE" and call(a4=0) == "PC_ERR_SHAPE"
    assert call(a9=ODD) == "PC_ERR_ALIGNMENT" and call(a10=P[3]) == "PC_ERR_UNSUPPORTED"
    for i in (4, 5, 6, 7, 8, 9):
        assert call(a7=_replace(st, i, 0)) == "PC_ERR_SHAPE"
    assert call(a0=0, a5=None) == "PC_OK"


def test_cpu_tensors_are_refused():
    x, i = torch.zeros(2, 4, 8), torch.zeros(2, dtype=torch.int32)
    pages = torch.zeros(3, 4, 2, 8)
    for fn, args in ((pc.qk_norm_rotary_fwd, (x, x)), (pc.qk_norm_rotary_bwd, (x, x, x, x)), (pc.attention_fwd, (x, x, x)),
                     (pc.attention_bwd, (x, x, x, x, x[0], x)), (pc.paged_attention, (x, pages, pages, i[None], i)),
                     (pc.paged_plan, (i, i, i[:, None], i, 4, 2)), (pc.paged_write, (x, x, pages, pages, i.long()))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            fn(*args)


def test_rotary_frequencies():
    f, a = pc.rotary_frequencies(8, device="cpu")
    want = torch.tensor([1.0, 0.1, 0.01, 0.001])
    assert a == 1.0 and torch.allclose(f, want, rtol=1e-6)
    f, a = pc.rotary_frequencies(8, factor=4, device="cpu")
    assert a == 1.0 and torch.allclose(f, want / 4, rtol=1e-6)
    f, a = pc.rotary_frequencies(8, factor=4, method="base", device="cpu")
    assert a == 1.0 and f[0] == 1 and f[-1].item() == pytest.approx(0.001 / 4, rel=1e-6)
    # turns over 4096 positions: 652, 65, 6.5, 0.65
    f, a = pc.rotary_frequencies(8, factor=4, method="bands", original=4096, device="cpu")
    kept = (4096 * 0.01 / (2 * math.pi) - 1) / 31
    assert a == pytest.approx(1 + 0.1 * math.log(4))
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01 * (kept + (1 - kept) / 4), 0.001 / 4]), rtol=1e-6)
    for bad in (dict(rotary=7), dict(rotary=0), dict(rotary=8, factor=0.5), dict(rotary=8, method="no"),
                dict(rotary=8, method="bands"), dict(rotary=8, base=-1.0)):
        with pytest.raises(ValueError):
            pc.rotary_frequencies(**bad, device="cpu")
