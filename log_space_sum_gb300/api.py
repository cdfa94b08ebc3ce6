"""PyTorch-facing wrappers of the C ABI: argument checks and marshalling only.

Every computation runs in libpcsum.so's CUDA kernels. PyTorch supplies device
memory (outputs and the scratch workspace) and the current CUDA stream.

Precision modes (pyjuice PR #62, Summary 1 table): "auto" (bf16 products),
"tf32" (TF32 products), "fp32" (3xTF32 products). The removed flags
``force_use_bf16`` / ``force_use_fp32`` raise a TypeError naming ``precision=``
when set to True and are accepted and ignored when False (same page, Breaking
change).
"""
from __future__ import annotations

import ctypes as C
import functools
import struct
import threading

import torch

from . import _native as N

PRECISIONS = {"auto": 0, "tf32": 1, "fp32": 2}

_local = threading.local()  # .workspaces: {(device, stream): buffer}, of this host thread


def precision_code(precision) -> int:
    if isinstance(precision, str):
        if precision not in PRECISIONS:
            raise ValueError(f"unknown precision {precision!r}; valid modes are 'auto' (bf16 "
                             "products), 'tf32' and 'fp32' (3xTF32)")
        return PRECISIONS[precision]
    if isinstance(precision, int) and not isinstance(precision, bool):
        return precision            # the library rejects unknown codes with PC_ERR_UNKNOWN_PRECISION
    raise TypeError(f"precision must be 'auto', 'tf32' or 'fp32', not {type(precision).__name__}")


def _removed_flags(kwargs: dict, where: str) -> None:
    for flag in ("force_use_bf16", "force_use_fp32"):
        if flag in kwargs:
            if kwargs.pop(flag):
                raise TypeError(f"{where}: {flag} was removed; pass precision='auto', 'tf32' or "
                                "'fp32' instead")
    if kwargs:
        raise TypeError(f"{where}: unexpected keyword arguments {sorted(kwargs)}")


def _check(t: torch.Tensor, name: str, dtype=torch.float32, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    # the handle alone: torch.cuda.current_stream would build a Stream object for each call
    if not isinstance(device, torch.device) or device.type != "cuda":
        return torch.cuda.current_stream(device).cuda_stream  # an index, a name, or its error
    index = device.index
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if index is None else index)


def workspace(nbytes: int, device) -> torch.Tensor:
    """Scratch buffer of at least nbytes, cached per (host thread, device, stream): the calls
    that share one run one after the other. Two threads' launches on one stream may alternate,
    so each has its own. A call that is being captured (torch.cuda.graph) takes one from the graph's
    own memory, which lasts as long as the graph and is no other call's: a cached one may be replaced
    before a replay, and replays are not ordered with the calls of the stream captured on."""
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    try:
        cache = _local.workspaces
    except AttributeError:
        cache = _local.workspaces = {}
    key = (device, _stream(device))
    ws = cache.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
        cache[key] = ws
    return ws


@functools.lru_cache(maxsize=4096)
def _query(name: str, *args) -> int:
    """A workspace size: a function of its arguments and of the GPU's SM count (one model
    of GPU per process)."""
    out = C.c_size_t(0)
    N.call(name, *args, C.byref(out))
    return out.value


# --------------------------------------------------------------------- sum layer
def sum_layer_fwd(theta, x, child_stride=None, precision="auto", out=None, **removed):
    """out[g,i,b] = m_b + log sum_j theta[g,i,j] exp(x[g*cs+j, b] - m_b) (pc_sum_layer_fwd)."""
    _removed_flags(removed, "sum_layer_fwd")
    prec = precision_code(precision)
    _check(theta, "theta")
    dev = theta.device
    _check(x, "x", device=dev)
    G, M, Nn = theta.shape
    B = x.shape[1]
    cs = (Nn if G > 1 else 0) if child_stride is None else int(child_stride)
    if out is None:
        out = torch.empty(G, M, B, dtype=torch.float32, device=dev)
    _check(out, "out", device=dev)
    nb = _query("pc_sum_layer_workspace", G, M, Nn, B, prec)
    ws = workspace(nb, dev)
    N.call("pc_sum_layer_fwd", G, M, Nn, B, _ptr(theta), _ptr(x), cs, _ptr(out), prec,
           _ptr(ws), ws.numel(), _stream(dev))
    return out


def sum_layer_bwd(theta, x, out, f, child_stride=None, precision="auto", element_flows=True,
                  param_flows=True, e=None, F=None, accumulate=False, **removed):
    """Element flows e (shaped like x) and parameter flows F (shaped like theta)
    (pc_sum_layer_bwd). Without ``accumulate`` the flows are overwritten; rows of x
    outside every group keep e's previous values (zeros for a fresh e)."""
    _removed_flags(removed, "sum_layer_bwd")
    prec = precision_code(precision)
    _check(theta, "theta")
    dev = theta.device
    for t, n in ((x, "x"), (out, "out"), (f, "f")):
        _check(t, n, device=dev)
    G, M, Nn = theta.shape
    B = x.shape[1]
    cs = (Nn if G > 1 else 0) if child_stride is None else int(child_stride)
    if element_flows and e is None:
        e = torch.zeros_like(x)
    if param_flows and F is None:
        F = torch.empty_like(theta)
    if e is not None:
        _check(e, "e", device=dev)
    if F is not None:
        _check(F, "F", device=dev)
    nb = _query("pc_sum_layer_workspace", G, M, Nn, B, prec)
    ws = workspace(nb, dev)
    N.call("pc_sum_layer_bwd", G, M, Nn, B, _ptr(theta), _ptr(x), cs, _ptr(out), _ptr(f),
           _ptr(e if element_flows else None), _ptr(F if param_flows else None), int(bool(accumulate)),
           prec, _ptr(ws), ws.numel(), _stream(dev))
    return (e if element_flows else None), (F if param_flows else None)


# --------------------------------------------------------------------------- HMM
def hmm_fwd_bwd(tokens, pi, A, E, precision="auto", flows=True, ll=None, dpi=None, dA=None, dE=None,
                accumulate=False, **removed):
    """Whole HMM circuit (pc_hmm_fwd_bwd): returns (ll [B] float64, dpi [H], dA [H,H],
    dE [H,V]); the flows are None when ``flows`` is False."""
    _removed_flags(removed, "hmm_fwd_bwd")
    prec = precision_code(precision)
    _check(A, "A")
    dev = A.device
    _check(tokens, "tokens", dtype=torch.int32, device=dev)
    _check(pi, "pi", device=dev)
    _check(E, "E", device=dev)
    B, T = tokens.shape
    H, V = E.shape
    if ll is None:
        ll = torch.empty(B, dtype=torch.float64, device=dev)
    _check(ll, "ll", dtype=torch.float64, device=dev)
    if flows:
        dpi = torch.empty(H, dtype=torch.float32, device=dev) if dpi is None else dpi
        dA = torch.empty(H, H, dtype=torch.float32, device=dev) if dA is None else dA
        dE = torch.empty(H, V, dtype=torch.float32, device=dev) if dE is None else dE
        for t, n in ((dpi, "dpi"), (dA, "dA"), (dE, "dE")):
            _check(t, n, device=dev)
    else:
        dpi = dA = dE = None
    nb = _query("pc_hmm_workspace", H, T, V, B, prec)
    ws = workspace(nb, dev)
    N.call("pc_hmm_fwd_bwd", H, T, V, B, _ptr(tokens), _ptr(pi), _ptr(A), _ptr(E), _ptr(ll),
           _ptr(dpi), _ptr(dA), _ptr(dE), int(bool(accumulate)), prec, _ptr(ws), ws.numel(),
           _stream(dev))
    return ll, dpi, dA, dE


def hmm_lowrank_fwd_bwd(tokens, pi, A, E, FA, FB, precision="auto", flows=True, accumulate=False, ll=None, dpi=None,
                        dA=None, W=None, dE=None, dFA=None, dFB=None, **removed):
    """HMM circuit with LowRank exp_sum transitions (pc_hmm_lowrank_fwd_bwd): FA
    [T-1,B,H,K], FB [T-1,B,K,H] the copies' factors. Returns a dict with ll [B] float64
    and, when ``flows``, dpi [H], dA [H,H] (sum of the copies' F+), W [H,H] (sum of their
    Z-correction statistics), dE [H,V], dFA, dFB (gradients of sum ll). Output tensors may
    be passed in (with ``accumulate`` the flows are added to them)."""
    _removed_flags(removed, "hmm_lowrank_fwd_bwd")
    prec = precision_code(precision)
    _check(A, "A")
    dev = A.device
    _check(tokens, "tokens", dtype=torch.int32, device=dev)
    for t, n in ((pi, "pi"), (E, "E"), (FA, "FA"), (FB, "FB")):
        _check(t, n, device=dev)
    B, T = tokens.shape
    H, V = E.shape
    K = FA.shape[-1]
    if tuple(FA.shape) != (max(T - 1, 0), B, H, K) or tuple(FB.shape) != (max(T - 1, 0), B, K, H):
        raise ValueError(f"FA {tuple(FA.shape)} and FB {tuple(FB.shape)}: expected [T-1,B,H,K] and [T-1,B,K,H]")
    out = dict(ll=torch.empty(B, dtype=torch.float64, device=dev) if ll is None else ll)
    _check(out["ll"], "ll", dtype=torch.float64, device=dev)
    if flows:
        new = lambda *shape: torch.empty(*shape, dtype=torch.float32, device=dev)  # noqa: E731
        given = dict(dpi=dpi, dA=dA, W=W, dE=dE, dFA=dFA, dFB=dFB)
        fresh = dict(dpi=lambda: new(H), dA=lambda: new(H, H), W=lambda: new(H, H), dE=lambda: new(H, V),
                     dFA=lambda: torch.empty_like(FA), dFB=lambda: torch.empty_like(FB))
        for k, v in given.items():
            out[k] = fresh[k]() if v is None else _check(v, k, device=dev)
    g = lambda k: _ptr(out.get(k))  # noqa: E731
    nb = _query("pc_hmm_lowrank_workspace", H, T, V, B, K, prec)
    ws = workspace(nb, dev)
    N.call("pc_hmm_lowrank_fwd_bwd", H, T, V, B, K, _ptr(tokens), _ptr(pi), _ptr(A), _ptr(E), _ptr(FA), _ptr(FB),
           g("ll"), g("dpi"), g("dA"), g("W"), g("dE"), g("dFA"), g("dFB"), int(bool(accumulate)), prec, _ptr(ws),
           ws.numel(), _stream(dev))
    return out


# -------------------------------------------------------------------------- HCLT
class HcltPrepared:
    """The HCLT's parameters in its contractions' formats (pc_hclt_prepare): reusable by
    every hclt_fwd_bwd call with the same tree, W, E and precision until they change."""

    def __init__(self, buf, parent, nvars, H, C, prec):
        self.buf, self.parent, self.nvars, self.H, self.C, self.prec = buf, parent, nvars, H, C, prec


def _host_parent(parent):
    import numpy as np
    return np.ascontiguousarray(np.asarray(parent.cpu() if isinstance(parent, torch.Tensor) else parent,
                                           dtype=np.int32))


def hclt_prepare(parent, W, E, precision="auto"):
    """Converts W and E once into the formats the HCLT's contractions read (pc_hclt_prepare)."""
    prec = precision_code(precision)
    _check(W, "W")
    dev = W.device
    _check(E, "E", device=dev)
    par = _host_parent(parent)
    n, H, Ccat = E.shape
    nb = _query("pc_hclt_prepare_bytes", n, H, Ccat, prec)
    buf = torch.empty(nb, dtype=torch.uint8, device=dev)
    N.call("pc_hclt_prepare", n, H, Ccat, par.ctypes.data_as(C.c_void_p), _ptr(W), _ptr(E), prec, _ptr(buf),
           buf.numel(), _stream(dev))
    return HcltPrepared(buf, par, n, H, Ccat, prec)


def hclt_fwd_bwd(parent, data, pi, W, E, precision="auto", flows=True, ll=None, dpi=None, dW=None, dE=None,
                 accumulate=False, prepared=None, **removed):
    """Whole HCLT circuit (pc_hclt_fwd_bwd). ``parent`` is a host int sequence
    (parent[0] = -1, parent[i] in [0, i)); data [B, nvars] int32 on the GPU; W
    [nvars, H, H]; E [nvars, H, C]. Returns (ll [B] float64, dpi, dW, dE). With
    ``prepared`` (from hclt_prepare for the same parent, W, E and precision) the call
    uses pc_hclt_fwd_bwd_prepared and E may be None."""
    import numpy as np

    _removed_flags(removed, "hclt_fwd_bwd")
    prec = precision_code(precision)
    _check(W, "W")
    dev = W.device
    _check(data, "data", dtype=torch.int32, device=dev)
    _check(pi, "pi", device=dev)
    par = _host_parent(parent)
    B, n = data.shape
    if prepared is not None:
        if prepared.prec != prec or prepared.nvars != n or not np.array_equal(prepared.parent, par):
            raise ValueError("prepared parameters were made for another tree or precision")
        H, Ccat = prepared.H, prepared.C
    else:
        _check(E, "E", device=dev)
        _, H, Ccat = E.shape
    if par.shape != (n,):
        raise ValueError(f"parent has shape {par.shape}, expected ({n},)")
    if ll is None:
        ll = torch.empty(B, dtype=torch.float64, device=dev)
    _check(ll, "ll", dtype=torch.float64, device=dev)
    if flows:
        dpi = torch.empty(H, dtype=torch.float32, device=dev) if dpi is None else dpi
        dW = torch.empty(n, H, H, dtype=torch.float32, device=dev) if dW is None else dW
        dE = torch.empty(n, H, Ccat, dtype=torch.float32, device=dev) if dE is None else dE
        for t, nm in ((dpi, "dpi"), (dW, "dW"), (dE, "dE")):
            _check(t, nm, device=dev)
    else:
        dpi = dW = dE = None
    if prepared is not None:
        nb = _query("pc_hclt_prepared_workspace", n, H, Ccat, B, prec)
        ws = workspace(nb, dev)
        N.call("pc_hclt_fwd_bwd_prepared", n, H, Ccat, B, par.ctypes.data_as(C.c_void_p), _ptr(data), _ptr(pi),
               _ptr(W), _ptr(prepared.buf), prepared.buf.numel(), _ptr(ll), _ptr(dpi), _ptr(dW), _ptr(dE),
               int(bool(accumulate)), prec, _ptr(ws), ws.numel(), _stream(dev))
        return ll, dpi, dW, dE
    nb = _query("pc_hclt_workspace", n, H, Ccat, B, prec)
    ws = workspace(nb, dev)
    N.call("pc_hclt_fwd_bwd", n, H, Ccat, B, par.ctypes.data_as(C.c_void_p), _ptr(data), _ptr(pi), _ptr(W), _ptr(E),
           _ptr(ll), _ptr(dpi), _ptr(dW), _ptr(dE), int(bool(accumulate)), prec, _ptr(ws), ws.numel(),
           _stream(dev))
    return ll, dpi, dW, dE


# ----------------------------------------------------------------------- LowRank
def _lowrank_shapes(theta, A, Bm, x):
    _check(theta, "theta")
    dev = theta.device
    for t, n in ((A, "A"), (Bm, "B"), (x, "x")):
        _check(t, n, device=dev)
    M, Nn = theta.shape
    Bs, Ma, K = A.shape
    if Ma != M or tuple(Bm.shape) != (Bs, K, Nn) or tuple(x.shape) != (Nn, Bs):
        raise ValueError(f"LowRank shapes: theta {tuple(theta.shape)}, A {tuple(A.shape)}, B {tuple(Bm.shape)}, "
                         f"x {tuple(x.shape)}; expected A [B,M,K], B [B,K,N], x [N,B]")
    return dev, M, Nn, K, Bs


def lowrank_exp_sum_fwd(theta, A, Bm, x, precision="auto", out=None, logZ=None, **removed):
    """LowRank exp_sum layer forward (pc_lowrank_exp_sum_fwd): returns out [M,B] and
    logZ [B,M] = log Z_b[i], which the backward reads."""
    _removed_flags(removed, "lowrank_exp_sum_fwd")
    prec = precision_code(precision)
    dev, M, Nn, K, Bs = _lowrank_shapes(theta, A, Bm, x)
    out = torch.empty(M, Bs, dtype=torch.float32, device=dev) if out is None else out
    logZ = torch.empty(Bs, M, dtype=torch.float32, device=dev) if logZ is None else logZ
    _check(out, "out", device=dev)
    _check(logZ, "logZ", device=dev)
    nb = _query("pc_lowrank_exp_sum_workspace", M, Nn, K, Bs, 0, prec)
    ws = workspace(nb, dev)
    N.call("pc_lowrank_exp_sum_fwd", M, Nn, K, Bs, _ptr(theta), _ptr(A), _ptr(Bm), _ptr(x), _ptr(out), _ptr(logZ),
           prec, _ptr(ws), ws.numel(), _stream(dev))
    return out, logZ


def lowrank_exp_sum_bwd(theta, A, Bm, x, out, logZ, f, precision="auto", grads=True, element_flows=True,
                        param_flows=True, z_correction=True, dA=None, dB=None, e=None, Fplus=None, W=None,
                        accumulate=False, **removed):
    """LowRank exp_sum layer backward (pc_lowrank_exp_sum_bwd): returns a dict with dA
    [B,M,K], dB [B,K,N] (``grads``), e [N,B] (``element_flows``), Fplus [M,N]
    (``param_flows``) and W [M,N] (``z_correction``); what is switched off is None."""
    _removed_flags(removed, "lowrank_exp_sum_bwd")
    prec = precision_code(precision)
    dev, M, Nn, K, Bs = _lowrank_shapes(theta, A, Bm, x)
    for t, n in ((out, "out"), (logZ, "logZ"), (f, "f")):
        _check(t, n, device=dev)
    new = lambda *shape: torch.empty(*shape, dtype=torch.float32, device=dev)  # noqa: E731
    dA = (new(Bs, M, K) if dA is None else dA) if grads else None
    dB = (new(Bs, K, Nn) if dB is None else dB) if grads else None
    e = (new(Nn, Bs) if e is None else e) if element_flows else None
    Fplus = (new(M, Nn) if Fplus is None else Fplus) if param_flows else None
    W = (new(M, Nn) if W is None else W) if z_correction else None
    for t, n in ((dA, "dA"), (dB, "dB"), (e, "e"), (Fplus, "Fplus"), (W, "W")):
        if t is not None:
            _check(t, n, device=dev)
    nb = _query("pc_lowrank_exp_sum_workspace", M, Nn, K, Bs, 1, prec)
    ws = workspace(nb, dev)
    N.call("pc_lowrank_exp_sum_bwd", M, Nn, K, Bs, _ptr(theta), _ptr(A), _ptr(Bm), _ptr(x), _ptr(out), _ptr(logZ),
           _ptr(f), _ptr(dA), _ptr(dB), _ptr(e), _ptr(Fplus), _ptr(W), int(bool(accumulate)), prec, _ptr(ws),
           ws.numel(), _stream(dev))
    return dict(dA=dA, dB=dB, e=e, Fplus=Fplus, W=W)


def lowrank_sum_exp_fwd(theta, A, Bm, x, precision="auto", out=None, logZ=None, **removed):
    """LowRank sum_exp layer forward (pc_lowrank_sum_exp_fwd), the scale g_b = exp(A_b)
    exp(B_b) summed over the rank: returns out [M,B] and logZ [B,M] = log Z_b[i]."""
    _removed_flags(removed, "lowrank_sum_exp_fwd")
    prec = precision_code(precision)
    dev, M, Nn, K, Bs = _lowrank_shapes(theta, A, Bm, x)
    out = torch.empty(M, Bs, dtype=torch.float32, device=dev) if out is None else out
    logZ = torch.empty(Bs, M, dtype=torch.float32, device=dev) if logZ is None else logZ
    _check(out, "out", device=dev)
    _check(logZ, "logZ", device=dev)
    nb = _query("pc_lowrank_sum_exp_workspace", M, Nn, K, Bs, 0, prec)
    ws = workspace(nb, dev)
    N.call("pc_lowrank_sum_exp_fwd", M, Nn, K, Bs, _ptr(theta), _ptr(A), _ptr(Bm), _ptr(x), _ptr(out), _ptr(logZ),
           prec, _ptr(ws), ws.numel(), _stream(dev))
    return out, logZ


def lowrank_sum_exp_bwd(theta, A, Bm, x, f, precision="auto", grads=True, element_flows=True, param_flows=True,
                        z_correction=True, dA=None, dB=None, e=None, Fplus=None, W=None, accumulate=False,
                        flow_precision="bf16", **removed):
    """LowRank sum_exp layer backward (pc_lowrank_sum_exp_bwd): the same outputs as
    lowrank_exp_sum_bwd (dA, dB, e, Fplus, W; what is switched off is None).
    ``flow_precision="fp8"`` (precision "auto"): Fplus and W from e4m3 products."""
    _removed_flags(removed, "lowrank_sum_exp_bwd")
    if flow_precision not in ("bf16", "fp8"):
        raise ValueError(f"flow_precision must be 'bf16' or 'fp8', got {flow_precision!r}")
    prec = precision_code(precision)
    dev, M, Nn, K, Bs = _lowrank_shapes(theta, A, Bm, x)
    _check(f, "f", device=dev)
    new = lambda *shape: torch.empty(*shape, dtype=torch.float32, device=dev)  # noqa: E731
    dA = (new(Bs, M, K) if dA is None else dA) if grads else None
    dB = (new(Bs, K, Nn) if dB is None else dB) if grads else None
    e = (new(Nn, Bs) if e is None else e) if element_flows else None
    Fplus = (new(M, Nn) if Fplus is None else Fplus) if param_flows else None
    W = (new(M, Nn) if W is None else W) if z_correction else None
    for t, n in ((dA, "dA"), (dB, "dB"), (e, "e"), (Fplus, "Fplus"), (W, "W")):
        if t is not None:
            _check(t, n, device=dev)
    nb = _query("pc_lowrank_sum_exp_workspace", M, Nn, K, Bs, 1, prec)
    ws = workspace(nb, dev)
    N.call("pc_lowrank_sum_exp_bwd", M, Nn, K, Bs, _ptr(theta), _ptr(A), _ptr(Bm), _ptr(x), _ptr(f), _ptr(dA),
           _ptr(dB), _ptr(e), _ptr(Fplus), _ptr(W), int(bool(accumulate)), int(flow_precision == "fp8"), prec,
           _ptr(ws), ws.numel(), _stream(dev))
    return dict(dA=dA, dB=dB, e=e, Fplus=Fplus, W=W)


# -------------------------------------------------------------------- EM M-step
def em_normalize(F: torch.Tensor, theta: torch.Tensor, W: torch.Tensor | None = None) -> torch.Tensor:
    """EM M-step (pc_em_normalize), in place on ``theta`` (shape [..., N], rows = nodes):
    theta = normalize(F) over the last axis, or with ``W`` the LowRank conditional update
    normalize(F / W) (0 where W <= 0). A row whose statistic sums to 0 keeps theta."""
    _check(F, "F")
    _check(theta, "theta", device=F.device)
    if W is not None:
        _check(W, "W", device=F.device)
    if F.shape != theta.shape or (W is not None and W.shape != F.shape):
        raise ValueError(f"F {tuple(F.shape)}, theta {tuple(theta.shape)} and W must have one shape")
    if F.dim() < 1 or F.numel() == 0:
        raise ValueError("F must have at least one element")
    Nn = F.shape[-1]
    rows = F.numel() // Nn
    N.call("pc_em_normalize", 1, rows, Nn, _ptr(F), _ptr(W), _ptr(theta), _stream(F.device))
    return theta


# --------------------------------------------------- the factor network's operators
# What a sequence model that supplies hmm_lowrank_fwd_bwd's factors FA, FB is made of, and
# what trains it from dFA, dFB. Elements are float32 or bfloat16.
DTYPES = {torch.float32: 0, torch.bfloat16: 1}


def _elements(t, name, dtype=None, device=None):
    """An activation: float32 or bfloat16 on the GPU, contiguous along its last dimension."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype not in DTYPES if dtype is None else t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype or 'torch.float32 or torch.bfloat16'}, got {t.dtype}")
    if t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _shaped(t, name, shape):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _rows(t, name):
    """(rows, row stride) of a tensor seen as rows of its last dimension."""
    if t.dim() == 2:
        return t.shape[0], t.stride(0)
    if t.is_contiguous():
        return (t.numel() // t.shape[-1] if t.shape[-1] else 0), t.shape[-1]
    try:
        flat = t.view(-1, t.shape[-1])
    except RuntimeError:
        raise ValueError(f"{name}'s leading dimensions must collapse to rows of one stride") from None
    return flat.shape[0], flat.stride(0)


def _param(t, name, dim, device):
    if t is not None:
        _shaped(_check(t, name, device=device), name, (dim,))
    return t


def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, out=None, mean=None, rstd=None):
    """Layer norm over the last dimension (pc_layer_norm_fwd): x [..., D] float32 or
    bfloat16, rows of any one stride; weight, bias [D] float32 or None. Returns (y, mean,
    rstd); the statistics [...] are float32 and what layer_norm_bwd reads."""
    _elements(x, "x")
    dev, D = x.device, (x.shape[-1] if x.dim() else 0)
    if D < 1:
        raise ValueError("x must have a last dimension of at least one")
    _param(weight, "weight", D, dev)
    _param(bias, "bias", D, dev)
    rows, ld = _rows(x, "x")
    out = torch.empty(x.shape, dtype=x.dtype, device=dev) if out is None else _shaped(
        _elements(out, "out", x.dtype, dev), "out", x.shape)
    lead = x.shape[:-1]
    mean = torch.empty(lead, dtype=torch.float32, device=dev) if mean is None else _shaped(
        _check(mean, "mean", device=dev), "mean", lead)
    rstd = torch.empty(lead, dtype=torch.float32, device=dev) if rstd is None else _shaped(
        _check(rstd, "rstd", device=dev), "rstd", lead)
    N.call("pc_layer_norm_fwd", rows, D, _ptr(x), ld, _ptr(weight), _ptr(bias), eps, _ptr(out),
           _rows(out, "out")[1], _ptr(mean), _ptr(rstd), DTYPES[x.dtype], _stream(dev))
    return out, mean, rstd


def layer_norm_bwd(dy, x, weight, mean, rstd, dx=None, dweight=None, dbias=None, params=True, accumulate=False):
    """Gradients of layer_norm_fwd (pc_layer_norm_bwd) from its statistics: returns (dx,
    dweight [D], dbias [D]), the last two float32 sums over all rows (None with ``params``
    False; added to the given tensors with ``accumulate``)."""
    _elements(x, "x")
    dev, D = x.device, (x.shape[-1] if x.dim() else 0)
    if D < 1:
        raise ValueError("x must have a last dimension of at least one")
    _shaped(_elements(dy, "dy", x.dtype, dev), "dy", x.shape)
    _param(weight, "weight", D, dev)
    for t, n in ((mean, "mean"), (rstd, "rstd")):
        _shaped(_check(t, n, device=dev), n, x.shape[:-1])
    if accumulate and params and (dweight is None or dbias is None):
        raise ValueError("accumulate needs dweight and dbias to add to")
    rows, ld = _rows(x, "x")
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev) if dx is None else _shaped(
        _elements(dx, "dx", x.dtype, dev), "dx", x.shape)
    ws, nb = None, 0
    if params:
        dweight = torch.empty(D, dtype=torch.float32, device=dev) if dweight is None else _param(
            dweight, "dweight", D, dev)
        dbias = torch.empty(D, dtype=torch.float32, device=dev) if dbias is None else _param(dbias, "dbias", D, dev)
        ws = workspace(_query("pc_layer_norm_bwd_workspace", rows, D), dev)
        nb = ws.numel()
    else:
        dweight = dbias = None
    N.call("pc_layer_norm_bwd", rows, D, _ptr(dy), _rows(dy, "dy")[1], _ptr(x), ld, _ptr(weight), _ptr(mean),
           _ptr(rstd), _ptr(dx), _rows(dx, "dx")[1], _ptr(dweight), _ptr(dbias), int(bool(accumulate)),
           DTYPES[x.dtype], _ptr(ws), nb, _stream(dev))
    return dx, dweight, dbias


def _strides(*tensors):
    flat = ()
    for t in tensors:
        flat += t.stride()[:-1]
    return struct.pack(f"{len(flat)}q", *flat)


def _attention_inputs(q, k, v, log_decay, state, lengths, lead):
    """Checks of q, k [*lead, H, Dk], v [*lead, H, Dv] and what goes with them."""
    _elements(q, "q")
    dev, dt = q.device, q.dtype
    if q.dim() != lead + 2:
        raise ValueError(f"q must have {lead + 2} dimensions, got {q.dim()}")
    H, Dk = q.shape[-2:]
    _shaped(_elements(k, "k", dt, dev), "k", q.shape)
    _elements(v, "v", dt, dev)
    if v.dim() != q.dim() or v.shape[:-1] != q.shape[:-1]:
        raise ValueError(f"v has shape {tuple(v.shape)}, expected {tuple(q.shape[:-1])} and a head size")
    Dv = v.shape[-1]
    _shaped(_check(log_decay, "log_decay", device=dev), "log_decay", (H,))
    if state is not None:
        _shaped(_check(state, "state", device=dev), "state", (q.shape[0], H, Dk, Dv))
    if lengths is not None:
        _shaped(_check(lengths, "lengths", dtype=torch.int32, device=dev), "lengths", (q.shape[0],))
    return dev, dt, H, Dk, Dv


def _given(t, name, shape, dtype, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _shaped(_elements(t, name, dtype, device), name, shape)


def linear_attention_fwd(q, k, v, log_decay, scale=1.0, state=None, lengths=None, out=None, state_out=None):
    """Linear attention with a decay for each head over whole sequences
    (pc_linear_attention_fwd): S_t = exp(log_decay) S_{t-1} + k_t v_t^T, o_t = scale q_t^T
    S_t. q, k [B,T,H,Dk], v [B,T,H,Dv] float32 or bfloat16, any strides with the last
    dimension contiguous; log_decay [H] <= 0, ``state`` [B,H,Dk,Dv] float32 (None: zeros),
    ``lengths`` [B] int32 (None: T). Returns (o [B,T,H,Dv], state after each sequence's
    last token). Outputs that are passed in may not overlap an input."""
    dev, dt, H, Dk, Dv = _attention_inputs(q, k, v, log_decay, state, lengths, 2)
    B, T = q.shape[:2]
    out = _given(out, "out", v.shape, dt, dev)
    if state_out is None:
        state_out = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=dev)
    _shaped(_check(state_out, "state_out", device=dev), "state_out", (B, H, Dk, Dv))
    code = DTYPES[dt]
    nb = _query("pc_linear_attention_workspace", B, T, H, Dk, Dv, 0, code)
    ws = workspace(nb, dev)
    N.call("pc_linear_attention_fwd", B, T, H, Dk, Dv, _ptr(q), _ptr(k), _ptr(v), _strides(q, k, v, out),
           _ptr(log_decay), scale, _ptr(state), _ptr(lengths), _ptr(out), _ptr(state_out), code, _ptr(ws),
           ws.numel(), _stream(dev))
    return out, state_out


def linear_attention_bwd(q, k, v, log_decay, do, scale=1.0, state=None, dstate=None, lengths=None, dq=None, dk=None,
                         dv=None, dstate_in=None):
    """Gradients of linear_attention_fwd (pc_linear_attention_bwd) from ``do`` [B,T,H,Dv]
    and, optionally, ``dstate`` [B,H,Dk,Dv], the gradient of the state it returned. Returns
    a dict with dq, dk, dv and dstate, the gradient of its initial state. dq, dk, dv may be
    passed in with any strides (slices of one projection's gradient); they and
    ``dstate_in``, where dstate is to lie, may not overlap an input or one another."""
    dev, dt, H, Dk, Dv = _attention_inputs(q, k, v, log_decay, state, lengths, 2)
    B, T = q.shape[:2]
    _shaped(_elements(do, "do", dt, dev), "do", v.shape)
    if dstate is not None:
        _shaped(_check(dstate, "dstate", device=dev), "dstate", (B, H, Dk, Dv))
    dq, dk, dv = (_given(t, n, like.shape, dt, dev)
                  for t, n, like in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)))
    if dstate_in is None:
        dstate_in = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=dev)
    _shaped(_check(dstate_in, "dstate_in", device=dev), "dstate_in", (B, H, Dk, Dv))
    code = DTYPES[dt]
    nb = _query("pc_linear_attention_workspace", B, T, H, Dk, Dv, 1, code)
    ws = workspace(nb, dev)
    N.call("pc_linear_attention_bwd", B, T, H, Dk, Dv, _ptr(q), _ptr(k), _ptr(v), _ptr(do),
           _strides(q, k, v, do, dq, dk, dv), _ptr(log_decay), scale, _ptr(state), _ptr(dstate), _ptr(lengths),
           _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dstate_in), code, _ptr(ws), ws.numel(), _stream(dev))
    return dict(dq=dq, dk=dk, dv=dv, dstate=dstate_in)


def linear_attention_step(q, k, v, log_decay, state, scale=1.0, out=None):
    """One token of each sequence (pc_linear_attention_step): q, k [B,H,Dk], v [B,H,Dv];
    ``state`` [B,H,Dk,Dv] float32 is updated in place. Returns o [B,H,Dv]."""
    dev, dt, H, Dk, Dv = _attention_inputs(q, k, v, log_decay, state, None, 1)
    if state is None:
        raise TypeError("state must be a torch.Tensor")
    out = _given(out, "out", v.shape, dt, dev)
    N.call("pc_linear_attention_step", q.shape[0], H, Dk, Dv, _ptr(q), _ptr(k), _ptr(v), _strides(q, k, v, out),
           _ptr(log_decay), scale, _ptr(state), _ptr(out), DTYPES[dt], _stream(dev))
    return out


def orthogonalize(G, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, precision="auto", out=None):
    """Orthogonalised update of a matrix or a stack of them (pc_orthogonalize): G [..., R,
    C] float32 or bfloat16, contiguous; ``steps`` Newton-Schulz products X <- a X + (b A +
    c A A) X, A = X X^T, from X = G / (|G|_F + eps). Returns X in G's shape and type.
    Operands have 11 significant bits with "auto" and "tf32", float32 G too: "fp32" (22 bits) for
    matrices of low rank, whose missing directions rounding fills and the iteration raises."""
    prec = precision_code(precision)
    _elements(G, "G")
    dev = G.device
    if G.dim() < 2:
        raise ValueError("G must have at least two dimensions")
    if not G.is_contiguous():
        raise ValueError("G must be contiguous")
    out = _given(out, "out", G.shape, G.dtype, dev)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    a, b, c = coefficients
    R, Cc = G.shape[-2:]
    if R < 1 or Cc < 1:
        raise ValueError("G's matrices must not be empty")
    batch = G.numel() // (R * Cc)
    ws = workspace(_query("pc_orthogonalize_workspace", batch, R, Cc, prec), dev)
    N.call("pc_orthogonalize", batch, R, Cc, _ptr(G), steps, a, b, c, eps, _ptr(out), DTYPES[G.dtype], prec,
           _ptr(ws), ws.numel(), _stream(dev))
    return out


# -------------------------------------------------------------------- diagnostics
def device_status(device=None) -> None:
    """Synchronises the current stream and raises PCError if a kernel gave up a bounded wait."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    N.call("pc_device_status", _stream(dev))


def set_wait_limit_ns(ns: int = 0) -> None:
    """Limit of the contraction kernel's first device-side waits on the current device
    (0 restores the 2 s default); a wait that runs out is reported by device_status()."""
    N.call("pc_set_wait_limit_ns", int(ns))


def profile_start(capacity: int = 4096) -> None:
    N.call("pc_profile_start", int(capacity))


def profile_stop(capacity: int = 4096):
    """Returns [(kind, ms, flops, launches)] for every record since profile_start: one
    contraction launch, or a chain of consecutive launches of one kind timed together."""
    cnt = C.c_int(0)
    ms = (C.c_float * capacity)()
    kind = (C.c_int * capacity)()
    flops = (C.c_longlong * capacity)()
    launches = (C.c_int * capacity)()
    N.call("pc_profile_stop", C.byref(cnt), ms, kind, flops, launches, int(capacity))
    return [(N.KINDS.get(kind[i], str(kind[i])), float(ms[i]), int(flops[i]), int(launches[i]))
            for i in range(cnt.value)]
