"""Operators of a factor network - the sequence model that supplies the LowRank factors of a
circuit's transition copies - as timed cases: layer norm (both directions), linear attention
with a decay for each head (prompt, its gradient, one token) and the orthogonalised update of
the network's weight matrices.

``run`` computes a case in plain float32 torch operations, or, with ``own`` true, through
this library's entry points on the same inputs. ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS_NORM = 1e-5
EPS_ORTH = 1e-7
STEPS = 5
COEF = (3.4445, -4.7750, 2.0315)
CHUNK = 128  # chunk of the plain linear attention


def _ln(name, way, rows, dim, dtype, bias=True):
    return dict(name=name, op="layer_norm", way=way, rows=rows, dim=dim, dtype=dtype, bias=bias)


def _la(name, way, batch, length, heads, dk, dv, dtype, state=False, ragged=False):
    return dict(name=name, op="linear_attention", way=way, batch=batch, length=length, heads=heads, dk=dk, dv=dv,
                dtype=dtype, state=state, ragged=ragged)


def _or(name, batch, m, n, dtype, precision):
    return dict(name=name, op="orthogonalize", way="fwd", batch=batch, m=m, n=n, dtype=dtype, precision=precision)


def listed():
    return [
        # one decoded position of a batch of 64: the call is launch and latency
        _ln("norm, 64 rows of 1024", "fwd", 64, 1024, "bf16"),
        # a training batch of 512 sequences of 64 positions, wide features: bandwidth
        _ln("norm, 32768 x 4096", "fwd", 32768, 4096, "bf16"),
        # the gradient of the same layer at 1024 features, with the weight's reduction
        _ln("norm gradient, 32768 x 1024", "bwd", 32768, 1024, "bf16"),
        # a ragged float32 gradient: odd row count, rows that are no multiple of 16 bytes
        _ln("norm gradient, 4097 x 1537", "bwd", 4097, 1537, "fp32"),
        # one token for each of 64 sequences: the states are read and written
        _la("attention step, 64 x 16 heads", "step", 64, 1, 16, 128, 128, "bf16", state=True),
        # prompts of several lengths padded to one batch, continuing a state
        _la("attention, 4 x 2000 ragged", "fwd", 4, 2000, 16, 128, 128, "bf16", state=True, ragged=True),
        # one long sequence: few heads to spread over the GPU, 257 chunks deep
        _la("attention, 1 x 32771", "fwd", 1, 32771, 16, 128, 128, "bf16"),
        # a training step's gradient
        _la("attention gradient, 8 x 2048", "bwd", 8, 2048, 16, 128, 128, "bf16"),
        # float32 activations, small odd heads, ragged, with the state's gradient
        _la("attention gradient, 3 x 333", "bwd", 3, 333, 5, 40, 56, "fp32", state=True, ragged=True),
        # a square weight of 1024 features
        _or("orthogonalise 1024 x 1024", 1, 1024, 1024, "bf16", "auto"),
        # the head that makes a copy's factor: 1024 features to 1024 latents x rank 16
        _or("orthogonalise 1024 x 16384", 1, 1024, 16384, "bf16", "auto"),
        # a stack of float32 weights, taller than wide, odd
        _or("orthogonalise 6 of 770 x 333", 6, 770, 333, "fp32", "fp32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["ln_fwd", "ln_bwd", "la_step", "la_fwd", "la_bwd", "orth"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if kind.startswith("ln"):
        dim = _log_int(rng, 64, 4096)
        if rng.random() < 0.6:
            dim = max(64, dim // 64 * 64)
        rows = _log_int(rng, 1, 32768 if dtype == "bf16" else 16384)
        c = _ln("", kind[3:], rows, dim, dtype, bias=rng.random() < 0.8)
    elif kind == "la_step":
        d = rng.choice([32, 64, 96, 128])
        c = _la("", "step", _log_int(rng, 1, 64), 1, rng.randint(2, 16), d, d, dtype, state=True)
    elif kind.startswith("la"):
        fp32 = dtype == "fp32"
        heads = rng.randint(2, 8 if fp32 else 16)
        dk = rng.choice([24, 40, 64] if fp32 else [64, 64, 72, 128, 128])
        dv = dk if rng.random() < 0.7 else rng.choice([48, 64] if fp32 else [64, 128])
        batch = rng.randint(1, 6)
        length = _log_int(rng, 1, (2048 if fp32 else 32768 if kind == "la_fwd" else 16384) // batch)
        c = _la("", kind[3:], batch, length, heads, dk, dv, dtype, state=rng.random() < 0.5, ragged=rng.random() < 0.4)
    else:
        fp32 = dtype == "fp32"
        m, n = _log_int(rng, 64, 768 if fp32 else 1024), _log_int(rng, 64, 1024 if fp32 else 8192)
        if rng.random() < 0.5:
            m, n = max(64, m // 64 * 64), max(64, n // 64 * 64)
        if rng.random() < 0.4:
            m, n = n, m
        batch = rng.choice([1, 1, 2, 4])
        if batch * m * n * min(m, n) > 1024 * 1024 * 16384:
            batch = 1
        c = _or("", batch, m, n, dtype, "fp32" if fp32 else "auto")
    del c["name"]
    return c


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    dt = _dtype(case)
    s = {"case": case}
    if case["op"] == "layer_norm":
        rows, dim = case["rows"], case["dim"]
        # a residual stream: features of different scale around a common offset
        s["x"] = (normal(rows, dim) * (0.5 + normal(dim).abs()) + 0.3).to(dt)
        s["weight"] = 1 + 0.2 * normal(dim)
        s["bias"] = 0.2 * normal(dim) if case["bias"] else None
        if case["way"] == "bwd":
            s["dy"] = (normal(rows, dim) + 0.1).to(dt)
            xf = s["x"].float()
            s["mean"] = xf.mean(-1)
            s["rstd"] = ((xf - s["mean"][:, None]).square().mean(-1) + EPS_NORM).rsqrt()
    elif case["op"] == "linear_attention":
        B, T, H, Dk, Dv = (case[k] for k in ("batch", "length", "heads", "dk", "dv"))
        # one projection's output, split into queries, keys and values without a copy
        proj = normal(B, T, H * (2 * Dk + Dv))
        proj[..., : 2 * H * Dk] *= Dk ** -0.25
        proj = proj.to(dt)
        s["q"], s["k"] = (proj[..., i * H * Dk:(i + 1) * H * Dk].unflatten(-1, (H, Dk)) for i in (0, 1))
        s["v"] = proj[..., 2 * H * Dk:].unflatten(-1, (H, Dv))
        # the heads' time constants run from 8 tokens to 2048
        s["log_decay"] = -torch.exp2(-3 - 8 * torch.arange(H, device=DEV) / max(1, H - 1)).float()
        s["scale"] = Dk ** -0.5
        s["state"] = normal(B, H, Dk, Dv) if case["state"] else None
        s["lengths"] = None
        if case["ragged"]:
            got = torch.randint(0, T + 1, (B,), generator=gen, device=DEV, dtype=torch.int32)
            got[0] = T
            s["lengths"] = got
        if case["way"] == "bwd":
            s["do"] = normal(B, T, H, Dv).to(dt)
            s["dstate"] = normal(B, H, Dk, Dv) if case["state"] else None
        if case["way"] == "step":
            s["q"], s["k"], s["v"] = s["q"][:, 0], s["k"][:, 0], s["v"][:, 0]
    else:
        m, n, batch = case["m"], case["n"], case["batch"]
        # a gradient: a few strong directions over a full-rank floor, at a gradient's size
        r = max(1, min(m, n) // 16)
        g = normal(batch, m, n) + normal(batch, m, r) @ normal(batch, r, n) / math.sqrt(r) * 2
        s["g"] = (g * 1e-3).to(dt)
    return s


def run(s):
    case = s["case"]
    return (_own if own else _plain)[case["op"] + "_" + case["way"]](s)


# ------------------------------------------------------------------------ plain forms
def _plain_layer_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    rstd = (c.square().mean(-1, keepdim=True) + EPS_NORM).rsqrt()
    y = c * rstd * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_layer_norm_bwd(s):
    dy = s["dy"].float()
    rstd = s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["weight"]
    dx = (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True)) * rstd
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}


def _chunked(x, n):
    """[B,T,H,D] -> float32 [B,H,n,CHUNK,D], zeros past T."""
    x = x.float().transpose(1, 2)
    x = torch.nn.functional.pad(x, (0, 0, 0, n * CHUNK - x.shape[2]))
    return x.unflatten(2, (n, CHUNK))


def _joined(x, T):
    return x.flatten(2, 3)[:, :, :T].transpose(1, 2)


class _Decays:
    """Powers of the heads' decays, over the tokens that are there."""

    def __init__(self, s):
        B, T = s["q"].shape[:2]
        self.T, self.n = T, -(-T // CHUNK)
        g = s["log_decay"]
        i = torch.arange(CHUNK, device=DEV)
        gap = (i[:, None] - i[None]).clamp(min=0)
        self.inner = torch.where(i[:, None] >= i, torch.exp(g[:, None, None] * gap), 0.0)[:, None]  # [H,1,C,C]
        self.after = torch.exp(g[:, None] * (i + 1))[:, None, :, None]           # lambda^(i+1)
        self.before = torch.exp(g[:, None] * (CHUNK - 1 - i))[:, None, :, None]  # lambda^(C-1-i)
        c = torch.arange(self.n, device=DEV)
        hop = (c[:, None] - c[None] - 1).clamp(min=0) * CHUNK
        self.outer = torch.where(c[:, None] > c, torch.exp(g[:, None, None] * hop), 0.0)  # [H,n,n]
        self.start = torch.exp(g[:, None] * (c * CHUNK))                                  # [H,n]
        t = torch.arange(T, device=DEV)
        self.len = torch.full((B,), T, device=DEV) if s["lengths"] is None else s["lengths"].long()
        there = t < self.len[:, None]
        self.there = there[:, :, None, None]                                              # [B,T,1,1]
        left = (self.len[:, None] - 1 - t).clamp(min=0)
        self.left = torch.where(there, torch.exp(g[:, None, None] * left), 0.0)           # [H,B,T]
        self.whole = torch.exp(g * self.len[:, None])[:, :, None, None]                   # [B,H,1,1]
        self.from_start = torch.exp(g[:, None] * (t + 1))                                 # [H,T]


def _start_states(d, k, v, state):
    """The state before each chunk: [B,H,n,Dk,Dv]."""
    u = (k * d.before).transpose(-1, -2) @ v
    at = (d.outer @ u.flatten(-2)).unflatten(-1, u.shape[-2:])
    return at if state is None else at + d.start[:, :, None, None] * state[:, :, None]


def _masked(x, d):
    return torch.where(d.there, x.float(), 0.0)


def _plain_linear_attention_fwd(s):
    d = _Decays(s)
    kt, vt = _masked(s["k"], d), _masked(s["v"], d)
    q, k, v = (_chunked(x, d.n) for x in (s["q"], kt, vt))
    at = _start_states(d, k, v, s["state"])
    o = ((q @ k.transpose(-1, -2)) * d.inner) @ v + (q * d.after) @ at
    o = torch.where(d.there, _joined(o, d.T) * s["scale"], 0.0)
    last = (kt * d.left.permute(1, 2, 0)[..., None]).permute(0, 2, 3, 1) @ vt.transpose(1, 2)
    if s["state"] is not None:
        last = last + d.whole * s["state"]
    return {"o": o.to(s["q"].dtype), "state": last}


def _plain_linear_attention_bwd(s):
    d = _Decays(s)
    qt, kt, vt, gt = (_masked(s[x], d) for x in ("q", "k", "v", "do"))
    q, k, v, g = (_chunked(x, d.n) for x in (qt, kt, vt, gt))
    scale, dt = s["scale"], s["q"].dtype
    at = _start_states(d, k, v, s["state"])
    p = (q @ k.transpose(-1, -2)) * d.inner
    dp = (g @ v.transpose(-1, -2)) * d.inner
    # what later chunks say of the state at a chunk's end
    ahead = (q * d.after).transpose(-1, -2) @ g
    ahead = (d.outer.transpose(-1, -2) @ ahead.flatten(-2)).unflatten(-1, ahead.shape[-2:])
    dq = dp @ k + (g * d.after) @ at.transpose(-1, -2)
    dk = dp.transpose(-1, -2) @ q + (v * d.before) @ ahead.transpose(-1, -2)
    dv = p.transpose(-1, -2) @ g + (k * d.before) @ ahead
    dq, dk, dv = (_joined(x, d.T) * scale for x in (dq, dk, dv))
    out = {}
    if s["state"] is not None:
        w = d.left.permute(1, 2, 0)[..., None]
        dk = dk + ((vt * w).transpose(1, 2) @ s["dstate"].transpose(-1, -2)).transpose(1, 2)
        dv = dv + ((kt * w).transpose(1, 2) @ s["dstate"]).transpose(1, 2)
        early = (qt * d.from_start.t()[None, :, :, None]).permute(0, 2, 3, 1) @ gt.transpose(1, 2)
        out["dstate"] = early * scale + d.whole * s["dstate"]
    return {**out, **{n: torch.where(d.there, x, 0.0).to(dt) for n, x in (("dq", dq), ("dk", dk), ("dv", dv))}}


def _plain_linear_attention_step(s):
    q, k, v = (s[x].float() for x in ("q", "k", "v"))
    new = torch.exp(s["log_decay"])[:, None, None] * s["state"] + k[..., :, None] * v[..., None, :]
    o = (q[..., None, :] @ new)[..., 0, :] * s["scale"]
    s["state"].copy_(new)
    return {"o": o.to(s["q"].dtype), "state": s["state"]}


def _plain_orthogonalize_fwd(s):
    x = s["g"].float()
    tall = x.shape[-2] > x.shape[-1]
    x = x.transpose(-1, -2) if tall else x
    x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + EPS_ORTH)
    a, b, c = COEF
    for _ in range(STEPS):  # the iteration itself
        y = x @ x.transpose(-1, -2)
        x = a * x + (b * y + c * (y @ y)) @ x
    return {"x": (x.transpose(-1, -2) if tall else x).to(s["g"].dtype)}


_plain = {
    "layer_norm_fwd": _plain_layer_norm_fwd,
    "layer_norm_bwd": _plain_layer_norm_bwd,
    "linear_attention_fwd": _plain_linear_attention_fwd,
    "linear_attention_bwd": _plain_linear_attention_bwd,
    "linear_attention_step": _plain_linear_attention_step,
    "orthogonalize_fwd": _plain_orthogonalize_fwd,
}


# ------------------------------------------------------------- the library's entry points
def _own_layer_norm_fwd(s):
    import log_space_sum_gb300 as pc
    y, mean, rstd = pc.layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=EPS_NORM)
    return {"y": y, "mean": mean, "rstd": rstd}


def _own_layer_norm_bwd(s):
    import log_space_sum_gb300 as pc
    dx, dweight, dbias = pc.layer_norm_bwd(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
    return {"dx": dx, "dweight": dweight, "dbias": dbias}


def _own_linear_attention_fwd(s):
    import log_space_sum_gb300 as pc
    o, state = pc.linear_attention_fwd(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"], state=s["state"],
                                       lengths=s["lengths"])
    return {"o": o, "state": state}


def _own_linear_attention_bwd(s):
    import log_space_sum_gb300 as pc
    got = pc.linear_attention_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"], scale=s["scale"],
                                  state=s["state"], dstate=s["dstate"], lengths=s["lengths"])
    out = {"dq": got["dq"], "dk": got["dk"], "dv": got["dv"]}
    if s["state"] is not None:
        out["dstate"] = got["dstate"]
    return out


def _own_linear_attention_step(s):
    import log_space_sum_gb300 as pc
    o = pc.linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"])
    return {"o": o, "state": s["state"]}


def _own_orthogonalize_fwd(s):
    import log_space_sum_gb300 as pc
    return {"x": pc.orthogonalize(s["g"], steps=STEPS, coefficients=COEF, eps=EPS_ORTH,
                                  precision=s["case"]["precision"])}


_own = {
    "layer_norm_fwd": _own_layer_norm_fwd,
    "layer_norm_bwd": _own_layer_norm_bwd,
    "linear_attention_fwd": _own_linear_attention_fwd,
    "linear_attention_bwd": _own_linear_attention_bwd,
    "linear_attention_step": _own_linear_attention_step,
    "orthogonalize_fwd": _own_orthogonalize_fwd,
}


# ------------------------------------------------------------------------ what it takes
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "layer_norm":
        rows, dim = case["rows"], case["dim"]
        if case["way"] == "fwd":  # x in, y out, the row statistics out, weight and bias in
            return {"bytes": 2 * rows * dim * es + 8 * rows + 8 * dim, "flops": 8 * rows * dim}
        return {"bytes": 3 * rows * dim * es + 8 * rows + 12 * dim, "flops": 13 * rows * dim}
    if case["op"] == "linear_attention":
        B, T, H, dk, dv = (case[k] for k in ("batch", "length", "heads", "dk", "dv"))
        tokens, states = B * T * H, B * H * dk * dv * 4
        if case["way"] == "bwd":  # q, k, v, do in, dq, dk, dv out; the two recurrences and three reads
            return {"bytes": tokens * es * (4 * dk + 3 * dv) + (3 * states if case["state"] else 0),
                    "flops": tokens * 10 * dk * dv}
        # q, k, v in, o out, the state in and out; the recurrence and its read
        return {"bytes": tokens * es * 2 * (dk + dv) + (2 if case["state"] else 1) * states,
                "flops": tokens * 4 * dk * dv}
    b, m, n = case["batch"], min(case["m"], case["n"]), max(case["m"], case["n"])
    # X X^T and its square are symmetric (half the products), then the product with X
    return {"bytes": 2 * b * m * n * es, "flops": STEPS * b * (3 * m * m * n + m * m * m)}


# ------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"] == "layer_norm":
        return _exact_norm(case, wide)
    if case["op"] == "linear_attention":
        return _exact_attention(case, wide)
    return _exact_orth(case, wide)


def _exact_norm(case, s):
    x = s["x"]
    if case["way"] == "fwd":
        var, mean = torch.var_mean(x, -1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS_NORM)
        y = (x - mean[:, None]) * rstd[:, None] * s["weight"]
        return {"y": y if s["bias"] is None else y + s["bias"], "mean": mean, "rstd": rstd}
    # the Jacobian of a normalised row, from the given statistics
    z = (x - s["mean"][:, None]) * s["rstd"][:, None]
    h = s["dy"] * s["weight"]
    n = x.shape[-1]
    dx = s["rstd"][:, None] / n * (n * h - h.sum(-1, keepdim=True) - z * (h * z).sum(-1, keepdim=True))
    return {"dx": dx, "dweight": torch.einsum("rd,rd->d", s["dy"], z), "dbias": s["dy"].sum(0)}


def _exact_attention(case, s):
    """The recurrences, one token after the other."""
    B, T, H, dk, dv = (case[k] for k in ("batch", "length", "heads", "dk", "dv"))
    lam = torch.exp(s["log_decay"])[:, None, None]
    S = torch.zeros(B, H, dk, dv, dtype=torch.float64, device=DEV) if s["state"] is None else s["state"].clone()
    if case["way"] == "step":
        S = lam * S + s["k"][..., None] * s["v"][..., None, :]
        return {"o": torch.einsum("bhk,bhkv->bhv", s["q"], S) * s["scale"], "state": S}
    n = torch.full((B,), T, device=DEV) if s["lengths"] is None else s["lengths"]
    here = (torch.arange(T, device=DEV) < n[:, None]).double()[:, :, None, None]  # [B,T,1,1]
    q, k, v = s["q"] * here, s["k"] * here, s["v"] * here
    keep = torch.where(here[..., None] > 0, lam, 1.0)  # [B,T,H,1,1]
    if case["way"] == "fwd":
        o = torch.zeros(B, T, H, dv, dtype=torch.float64, device=DEV)
        for t in range(T):
            S.mul_(keep[:, t]).add_(k[:, t, :, :, None] * v[:, t, :, None, :])
            o[:, t] = (q[:, t, :, None, :] @ S)[:, :, 0] * s["scale"]
        return {"o": o, "state": S}
    g = s["do"] * here
    dq, dkk, dvv = (torch.zeros_like(x) for x in (q, k, v))
    for t in range(T):
        S.mul_(keep[:, t]).add_(k[:, t, :, :, None] * v[:, t, :, None, :])
        dq[:, t] = (S @ g[:, t, :, :, None])[..., 0] * s["scale"]
    R = torch.zeros_like(S) if s.get("dstate") is None else s["dstate"].clone()
    for t in reversed(range(T)):
        R.add_(q[:, t, :, :, None] * g[:, t, :, None, :] * s["scale"])
        dkk[:, t] = (R @ v[:, t, :, :, None])[..., 0]
        dvv[:, t] = (k[:, t, :, None, :] @ R)[:, :, 0]
        R.mul_(keep[:, t])
    out = {"dq": dq, "dk": dkk * here, "dv": dvv * here}
    if s["state"] is not None:
        out["dstate"] = R
    return out


def _exact_orth(case, s):
    x = s["g"]
    b, m, n = x.shape
    if 2.0 * b * STEPS * min(m, n) ** 2 * (2 * max(m, n) + min(m, n)) > 1.5e13:
        return None
    x = x / (torch.linalg.norm(x.flatten(1), dim=1)[:, None, None] + EPS_ORTH)
    ca, cb, cc = COEF
    for _ in range(STEPS):
        if m <= n:
            y = torch.einsum("bij,bkj->bik", x, x)
            x = ca * x + cb * (y @ x) + cc * (y @ (y @ x))
        else:
            y = torch.einsum("bji,bjk->bik", x, x)
            x = ca * x + cb * (x @ y) + cc * ((x @ y) @ y)
    return {"x": x}
