"""Operators of a factor network whose layers look back by softmax attention, as timed cases:
norms of queries and keys with the rotation by position (both directions), causal attention
over packed prompts (both directions), attention of new tokens over a paged cache, and that
cache's tables, slots and writes.

``run`` computes a case in plain torch operations in 32 bits (angles in 64), or, with ``own``
true, through this library's entry points on the same inputs. ``exact`` is the definition in
64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
ROWS = 2048  # rows of scores that the plain form holds at once


def _rot(name, way, tokens, heads, kv_heads, dim, rotary, layout, dtype, far=False, norm=True):
    return dict(name=name, op="qk_norm_rotary", way=way, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim,
                rotary=rotary, layout=layout, dtype=dtype, far=far, norm=norm)


def _att(name, way, batch, longest, heads, kv_heads, dim, dtype, ragged=False):
    return dict(name=name, op="attention", way=way, batch=batch, longest=longest, heads=heads, kv_heads=kv_heads, dim=dim,
                dtype=dtype, ragged=ragged)


def _paged(name, batch, longest, new, page, heads, kv_heads, dim, dtype, ragged=False):
    return dict(name=name, op="paged_attention", way="fwd", batch=batch, longest=longest, new=new, page=page, heads=heads,
                kv_heads=kv_heads, dim=dim, dtype=dtype, ragged=ragged)


def _cache(name, batch, longest, new, page, kv_heads, dim, dtype, ragged=False):
    return dict(name=name, op="paged_cache", way="fwd", batch=batch, longest=longest, new=new, page=page,
                kv_heads=kv_heads, dim=dim, dtype=dtype, ragged=ragged)


def listed():
    return [
        # one token for each of 64 sequences in the middle of long ones: launch and latency
        _rot("norm + rotation, 64 tokens", "fwd", 64, 32, 8, 128, 128, "half", "bf16", far=True),
        # a batch of prompts, a quarter of the head left as it is: bandwidth
        _rot("norm + rotation, 32768 tokens", "fwd", 32768, 16, 2, 128, 96, "interleaved", "bf16"),
        # a training step's gradient, with the norms' weights
        _rot("norm + rotation gradient, 16384 tokens", "bwd", 16384, 16, 2, 128, 128, "half", "bf16"),
        # a training batch of equal sequences
        _att("attention, 8 x 2048", "fwd", 8, 2048, 16, 2, 128, "bf16"),
        # one long prompt
        _att("attention, 1 x 32771", "fwd", 1, 32771, 16, 2, 128, "bf16"),
        # the gradient of packed sequences of different lengths
        _att("attention gradient, 12 to 4096", "bwd", 12, 4096, 16, 2, 128, "bf16", ragged=True),
        # float32 activations, small odd heads, short sequences
        _att("attention gradient, 3 to 333", "bwd", 3, 333, 6, 3, 40, "fp32", ragged=True),
        # one token for each of 64 sequences of different lengths
        _paged("paged attention, 64 to 8192", 64, 8192, 1, 16, 32, 8, 128, "bf16", ragged=True),
        # one token of a single long sequence: the whole GPU reads one cache
        _paged("paged attention, 1 x 131072", 1, 131072, 1, 64, 32, 8, 128, "bf16"),
        # four prompts continued by a chunk each
        _paged("paged attention, 4 chunks of 512", 4, 8192, 512, 32, 16, 2, 128, "bf16", ragged=True),
        # the cache's bookkeeping and writes for one token each
        _cache("paged cache, 64 tokens", 64, 8192, 1, 16, 8, 128, "bf16", ragged=True),
        # ... and for whole prompts
        _cache("paged cache, 16 prompts", 16, 4096, 4096, 64, 8, 128, "bf16", ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rot_fwd", "rot_bwd", "att_fwd", "att_bwd", "paged", "paged", "cache"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    fp32 = dtype == "fp32"
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
    dim = rng.choice([40, 64, 80] if fp32 else [64, 64, 72, 96, 128, 128, 128])
    ragged = rng.random() < 0.6
    if kind.startswith("rot"):
        tokens = _log_int(rng, 1, max(16, min(32768, (1 << 26) // (dim * (heads + kv_heads)))))
        c = _rot("", kind[4:], tokens, heads, kv_heads, dim, dim if rng.random() < 0.5 else rng.randint(1, dim // 2) * 2,
                 rng.choice(["half", "interleaved"]), dtype, rng.random() < 0.5, rng.random() < 0.8)
    elif kind.startswith("att"):
        batch = rng.randint(1, 12)
        heads = min(heads, 16 // kv_heads * kv_heads)
        longest = _log_int(rng, 1, (2048 if fp32 else 16384 if kind == "att_fwd" else 8192) // batch)
        c = _att("", kind[4:], batch, longest, heads, kv_heads, dim, dtype, ragged)
    elif kind == "paged":
        batch = _log_int(rng, 1, 64)
        longest = _log_int(rng, 1, (16384 if fp32 else 131072) // batch)
        new = min(longest, rng.choice([1, 1, 1, 2, 5, 17, 64, 200, 512]))
        while new > 1 and batch * new * heads > 32768:
            new //= 2
        c = _paged("", batch, longest, new, rng.choice([16, 32, 48, 64, 128]), heads, kv_heads, dim, dtype, ragged)
    else:
        batch = _log_int(rng, 1, 256)
        longest = _log_int(rng, 1, 65536 // batch)
        c = _cache("", batch, longest, min(longest, rng.choice([1, 1, 7, 300, 4096])), rng.choice([16, 32, 64, 128]), kv_heads,
                   dim, dtype, ragged)
    del c["name"]
    return c


def _lengths(case):
    """Lengths of a case's sequences: the same for every seed."""
    n, top = case["batch"], case["longest"]
    if not case["ragged"]:
        return [top] * n
    rng = random.Random(n * 1000003 + top)
    return [top] + [rng.randint(1, top) for _ in range(n - 1)]


def _new(case):
    """New tokens of each sequence, the last ones of its length."""
    return [min(case["new"], n) for n in _lengths(case)]


def _starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    dt, D, Hk = _dtype(case), case["dim"], case["kv_heads"]
    H = case.get("heads", 0)
    s = {"case": case}

    def projected(T):
        """Queries, keys and values as slices of one projection's output."""
        proj = (normal(T, (H + 2 * Hk) * D)).to(dt)
        return (proj[:, :H * D].unflatten(-1, (H, D)), proj[:, H * D:(H + Hk) * D].unflatten(-1, (Hk, D)),
                proj[:, (H + Hk) * D:].unflatten(-1, (Hk, D)))

    if case["op"] == "qk_norm_rotary":
        T, R = case["tokens"], case["rotary"]
        s["q"], s["k"], _ = projected(T)
        s["q_weight"], s["k_weight"] = (1 + 0.2 * normal(D) if case["norm"] else None for _ in range(2))
        # tokens of sequences that have come far, or prompts of 2048 tokens one after the other
        s["positions"] = (torch.randint(0, 131072, (T,), generator=gen, device=DEV) if case["far"]
                          else torch.arange(T, device=DEV) % 2048).to(torch.int32)
        s["frequencies"] = (10000.0 ** (-torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)).float()
        if case["way"] == "bwd":
            s["dq"], s["dk"] = (normal(T, h, D).to(dt) for h in (H, Hk))
        return s
    lengths = _lengths(case)
    if case["op"] == "attention":
        T = sum(lengths)
        s["lengths"], s["starts"] = lengths, _ints(_starts(lengths))
        s["q"], s["k"], s["v"] = projected(T)
        s["scale"] = D ** -0.5
        if case["way"] == "bwd":
            out = _plain_attention_fwd(s)  # what the forward left
            s["o"], s["lse"] = out["o"], out["lse"]
            s["do"] = normal(T, H, D).to(dt)
        return s
    # a paged cache: its pages lie in no order
    page, new = case["page"], _new(case)
    cached = [n - m for n, m in zip(lengths, new)]
    width = -(-case["longest"] // page) + 3
    pages = sum(-(-n // page) for n in lengths) + 5
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).tolist()
    s["lengths"], s["new"], s["starts"] = lengths, new, _ints(_starts(new))
    T = sum(new)
    s["q"], s["k"], s["v"] = projected(T)
    s["k_pages"], s["v_pages"] = (normal(pages, page, Hk, D).to(dt) for _ in range(2))
    held = lengths if case["op"] == "paged_attention" else cached
    tables, at = torch.full((case["batch"], width), -1, dtype=torch.int32), 0
    for b, n in enumerate(held):
        need = -(-n // page)
        tables[b, :need] = torch.tensor(order[at:at + need], dtype=torch.int32)
        at += need
    s["tables"] = tables.to(DEV)
    if case["op"] == "paged_attention":
        s["total"], s["scale"] = _ints(lengths), D ** -0.5
    else:
        s["cached"], s["added"], s["free"] = _ints(cached), _ints(new), _ints(order[at:])
    return s


def run(s):
    case = s["case"]
    return (_own if own else _plain)[case["op"] + "_" + case["way"]](s)


# ------------------------------------------------------------------------ plain forms
def _angles(s):
    """cos and sin of the positions' angles: 64 bits, as far positions pass what 32 hold."""
    a = s["positions"].double()[:, None] * s["frequencies"].double()
    return a.cos().float()[:, None], a.sin().float()[:, None]  # [T,1,R/2]


def _halves(x, case):
    R = case["rotary"]
    if case["layout"] == "half":
        return x[..., :R // 2], x[..., R // 2:R]
    return x[..., 0:R:2], x[..., 1:R:2]


def _rotated(x, cos, sin, case):
    y = x.clone()
    a, b = _halves(x, case)
    c, d = _halves(y, case)
    c.copy_(a * cos - b * sin)
    d.copy_(b * cos + a * sin)
    return y


def _plain_rotary_fwd(s):
    case = s["case"]
    cos, sin = _angles(s)
    out = {}
    for n in ("q", "k"):
        x = s[n].float()
        if case["norm"]:
            x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * s[n + "_weight"]
        out[n] = _rotated(x, cos, sin, case).to(s[n].dtype)
    return out


def _plain_rotary_bwd(s):
    case = s["case"]
    cos, sin = _angles(s)
    out = {}
    for n in ("q", "k"):
        g = _rotated(s["d" + n].float(), cos, -sin, case)
        if case["norm"]:
            x, w = s[n].float(), s[n + "_weight"]
            rstd = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
            z = x * rstd
            out["d" + n + "_weight"] = (g * z).sum((0, 1))
            g = g * w
            g = rstd * (g - z * (g * z).mean(-1, keepdim=True))
        out["d" + n] = g.to(s[n].dtype)
    return out


def _visible(q, k, scale, before):
    """Scores of rows q [h,n,D], row i at position before + i, over keys k [h,m,D]."""
    p = (q @ k.transpose(-1, -2)) * scale
    i = torch.arange(q.shape[1], device=DEV) + before
    return p.masked_fill(torch.arange(k.shape[1], device=DEV) > i[:, None], float("-inf"))


def _head_major(x, group=1):
    return x.float().transpose(0, 1).repeat_interleave(group, 0)


def _plain_attend(q, k, v, scale, before):
    """Rows of one sequence and group of heads: (o, log of the sum)."""
    o, lse = [], []
    for r in range(0, q.shape[1], ROWS):
        at = q[:, r:r + ROWS]
        top = before + r + at.shape[1]
        p = _visible(at, k[:, :top], scale, before + r)
        m = p.amax(-1, keepdim=True)
        p = (p - m).exp()
        z = p.sum(-1, keepdim=True)
        o.append((p @ v[:, :top]) / z)
        lse.append((m + z.log())[..., 0])
    return torch.cat(o, 1), torch.cat(lse, 1)


def _plain_attention_fwd(s):
    q, k, v = s["q"], s["k"], s["v"]
    group = q.shape[1] // k.shape[1]
    o, lse, at = torch.empty(q.shape, dtype=q.dtype, device=DEV), torch.empty(q.shape[1], q.shape[0], device=DEV), 0
    for n in s["lengths"]:
        for h in range(k.shape[1]):  # a group of heads at a time: its scores fit
            hs, ts = slice(h * group, (h + 1) * group), slice(at, at + n)
            x, z = _plain_attend(_head_major(q[ts, hs]), _head_major(k[ts, h:h + 1]), _head_major(v[ts, h:h + 1]), s["scale"], 0)
            o[ts, hs] = x.transpose(0, 1).to(o.dtype)
            lse[hs, ts] = z
        at += n
    return {"o": o, "lse": lse}


def _plain_attention_bwd(s):
    q, k, v, do = (s[n] for n in ("q", "k", "v", "do"))
    group, scale, at = q.shape[1] // k.shape[1], s["scale"], 0
    delta = (do.float() * s["o"].float()).sum(-1)
    dq, dk, dv = (torch.zeros(x.shape, dtype=x.dtype, device=DEV) for x in (q, k, v))
    for n in s["lengths"]:
        for h in range(k.shape[1]):
            hs, ts = slice(h * group, (h + 1) * group), slice(at, at + n)
            Q, G = _head_major(q[ts, hs]), _head_major(do[ts, hs])
            K, V = _head_major(k[ts, h:h + 1]), _head_major(v[ts, h:h + 1])
            gq, gk, gv = torch.empty_like(Q), torch.zeros_like(K), torch.zeros_like(V)
            for r in range(0, n, ROWS):
                rs = slice(r, min(r + ROWS, n))
                top = rs.stop
                p = (_visible(Q[:, rs], K[:, :top], scale, r) - s["lse"][hs, at + r:at + top, None]).exp()
                ds = p * (G[:, rs] @ V[:, :top].transpose(-1, -2) - delta[at + r:at + top, hs].t()[..., None])
                gq[:, rs] = ds @ K[:, :top] * scale
                gk[0, :top] += (ds.transpose(-1, -2) @ Q[:, rs]).sum(0) * scale
                gv[0, :top] += (p.transpose(-1, -2) @ G[:, rs]).sum(0)
            dq[ts, hs] = gq.transpose(0, 1).to(dq.dtype)
            dk[ts, h], dv[ts, h] = gk[0].to(dk.dtype), gv[0].to(dv.dtype)
        at += n
    return {"dq": dq, "dk": dk, "dv": dv}


def _plain_paged_attention_fwd(s):
    q, page = s["q"], s["case"]["page"]
    group = q.shape[1] // s["k_pages"].shape[2]
    o, at = torch.empty(q.shape, dtype=q.dtype, device=DEV), 0
    for b, (n, m) in enumerate(zip(s["lengths"], s["new"])):
        held = s["tables"][b, :-(-n // page)].long()
        k, v = (_head_major(s[x][held].flatten(0, 1)[:n], group) for x in ("k_pages", "v_pages"))
        o[at:at + m] = _plain_attend(_head_major(q[at:at + m]), k, v, s["scale"], n - m)[0].transpose(0, 1).to(o.dtype)
        at += m
    return {"o": o}


def _plain_paged_cache_fwd(s):
    page, cached, added, tables = s["case"]["page"], s["cached"].long(), s["added"].long(), s["tables"]
    T, B = s["k"].shape[0], cached.shape[0]
    have, want = (cached + page - 1) // page, (cached + added + page - 1) // page
    first = (want - have).cumsum(0) - (want - have)
    col = torch.arange(tables.shape[1], device=DEV)
    fresh = (col >= have[:, None]) & (col < want[:, None])
    at = (first - have)[:, None] + col
    tables.copy_(torch.where(fresh, s["free"][at.clamp(0, s["free"].shape[0] - 1)], tables))
    starts = torch.cat([added.new_zeros(1), added.cumsum(0)])
    token = torch.arange(T, device=DEV)
    seq = (torch.searchsorted(starts, token, right=True) - 1).clamp(0, B - 1)
    positions = cached[seq] + token - starts[seq]
    slots = tables[seq, positions // page].long() * page + positions % page
    for n in ("k", "v"):
        s[n + "_pages"].flatten(0, 1)[slots] = s[n]
    return {"starts": starts.int(), "lengths": (cached + added).int(), "positions": positions.int(), "slots": slots,
            "taken": (want - have).sum(0, keepdim=True).int(), "tables": tables, "k_pages": s["k_pages"],
            "v_pages": s["v_pages"]}


_plain = {
    "qk_norm_rotary_fwd": _plain_rotary_fwd,
    "qk_norm_rotary_bwd": _plain_rotary_bwd,
    "attention_fwd": _plain_attention_fwd,
    "attention_bwd": _plain_attention_bwd,
    "paged_attention_fwd": _plain_paged_attention_fwd,
    "paged_cache_fwd": _plain_paged_cache_fwd,
}


# ------------------------------------------------------------- the library's entry points
def _own_rotary_fwd(s):
    import log_space_sum_gb300 as pc
    c = s["case"]
    q, k = pc.qk_norm_rotary_fwd(s["q"], s["k"], s["positions"], s["frequencies"], s["q_weight"], s["k_weight"], eps=EPS,
                                 layout=c["layout"], norm=c["norm"])
    return {"q": q, "k": k}


def _own_rotary_bwd(s):
    import log_space_sum_gb300 as pc
    c = s["case"]
    got = pc.qk_norm_rotary_bwd(s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["frequencies"], s["q_weight"],
                                s["k_weight"], eps=EPS, layout=c["layout"], norm=c["norm"])
    names = ("dq", "dk", "dq_weight", "dk_weight") if c["norm"] else ("dq", "dk")
    return {n: got[n] for n in names}


def _own_attention_fwd(s):
    import log_space_sum_gb300 as pc
    o, lse = pc.attention_fwd(s["q"], s["k"], s["v"], starts=s["starts"], scale=s["scale"])
    return {"o": o, "lse": lse}


def _own_attention_bwd(s):
    import log_space_sum_gb300 as pc
    return pc.attention_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], starts=s["starts"], scale=s["scale"])


def _own_paged_attention_fwd(s):
    import log_space_sum_gb300 as pc
    return {"o": pc.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["tables"], s["total"], starts=s["starts"],
                                    scale=s["scale"])}


def _own_paged_cache_fwd(s):
    import log_space_sum_gb300 as pc
    plan = pc.paged_plan(s["cached"], s["added"], s["tables"], s["free"], page_size=s["case"]["page"],
                         tokens=s["k"].shape[0])
    pc.paged_write(s["k"], s["v"], s["k_pages"], s["v_pages"], plan["slots"])
    return {**{n: plan[n] for n in ("starts", "lengths", "positions", "slots", "taken")}, "tables": s["tables"],
            "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


_own = {
    "qk_norm_rotary_fwd": _own_rotary_fwd,
    "qk_norm_rotary_bwd": _own_rotary_bwd,
    "attention_fwd": _own_attention_fwd,
    "attention_bwd": _own_attention_bwd,
    "paged_attention_fwd": _own_paged_attention_fwd,
    "paged_cache_fwd": _own_paged_cache_fwd,
}


# ------------------------------------------------------------------------ what it takes
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    D, Hk = case["dim"], case["kv_heads"]
    H = case.get("heads", Hk)
    if case["op"] == "qk_norm_rotary":
        n = case["tokens"] * (H + Hk) * D
        if case["way"] == "fwd":  # in and out; square and sum, two products, the rotation
            return {"bytes": 2 * n * es + 4 * case["tokens"], "flops": 7 * n}
        # gradient in, x in where there is a norm, gradient out
        return {"bytes": (3 if case["norm"] else 2) * n * es + 4 * case["tokens"], "flops": 14 * n}
    lengths = _lengths(case)
    if case["op"] == "attention":
        T, pairs = sum(lengths), sum(n * (n + 1) // 2 for n in lengths)
        if case["way"] == "fwd":  # q, k, v in, o and the rows' logarithms out; two products
            return {"bytes": T * D * es * 2 * (H + Hk) + 4 * T * H, "flops": 4 * D * H * pairs}
        # q, k, v, o, do and the logarithms in, three gradients out; five products
        return {"bytes": T * D * es * (4 * H + 4 * Hk) + 4 * T * H, "flops": 10 * D * H * pairs}
    new = _new(case)
    T = sum(new)
    if case["op"] == "paged_attention":
        pairs = sum(m * n - m * (m - 1) // 2 for n, m in zip(lengths, new))
        return {"bytes": 2 * sum(lengths) * Hk * D * es + 2 * T * H * D * es, "flops": 4 * D * H * pairs}
    return {"bytes": 4 * T * Hk * D * es + 12 * T + 16 * case["batch"], "flops": 4 * T}


# ------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "paged_cache":
        return _exact_cache(case, s)
    wide = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"] == "qk_norm_rotary":
        return _exact_rotary(case, wide)
    if work(case)["flops"] > 5e12:
        return None
    return _exact_paged(case, wide) if case["op"] == "paged_attention" else _exact_attention(case, wide)


def _exact_rotary(case, s):
    """The rotation as a product of complex numbers."""
    R, half = case["rotary"], case["layout"] == "half"
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), torch.outer(s["positions"].double(), s["frequencies"]))[:, None]

    def rotate(x, by):
        z = torch.complex(*(x[..., :R].unflatten(-1, (2, R // 2)).unbind(-2) if half
                            else x[..., :R].unflatten(-1, (R // 2, 2)).unbind(-1))) * by
        z = torch.stack([z.real, z.imag], -2 if half else -1).flatten(-2)
        return torch.cat([z, x[..., R:]], -1)

    out = {}
    for n in ("q", "k"):
        x = s[n]
        inv = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + EPS)
        if case["way"] == "fwd":
            out[n] = rotate(x * inv * s[n + "_weight"] if case["norm"] else x, turn)
            continue
        g = rotate(s["d" + n], turn.conj())
        if case["norm"]:
            out["d" + n + "_weight"] = torch.einsum("thd,thd->d", g, x * inv)
            u = g * s[n + "_weight"]
            g = inv * u - x * inv ** 3 * (u * x).sum(-1, keepdim=True) / case["dim"]
        out["d" + n] = g
    return out


def _exact_blocks(n, m, H):
    """Rows of a sequence's last m positions, so many at a time that H heads' scores fit."""
    step = max(1, min(m, (1 << 28) // max(1, n * H)))
    return [(r, min(r + step, m)) for r in range(0, m, step)]


def _exact_attention(case, s):
    H, Hk, scale, at = case["heads"], case["kv_heads"], s["scale"], 0
    g = H // Hk
    o, lse = torch.zeros_like(s["q"]), s["q"].new_zeros(H, s["q"].shape[0])
    dq, dk, dv = (torch.zeros_like(s[x]) for x in ("q", "k", "v"))
    for n in s["lengths"]:
        k, v = s["k"][at:at + n], s["v"][at:at + n]
        for a, b in _exact_blocks(n, n, H):
            rows = slice(at + a, at + b)
            q = s["q"][rows].unflatten(1, (Hk, g))
            w = torch.einsum("ihgd,jhd->hgij", q, k[:b]) * scale
            w.masked_fill_(torch.ones(b - a, b, dtype=torch.bool, device=DEV).triu(a + 1), -math.inf)
            z = torch.logsumexp(w, -1, keepdim=True)
            w = torch.exp(w - z)
            out = torch.einsum("hgij,jhd->ihgd", w, v[:b])
            o[rows], lse[:, rows] = out.flatten(1, 2), z[..., 0].flatten(0, 1)
            if case["way"] == "bwd":
                do = s["do"][rows].unflatten(1, (Hk, g))
                dv[at:at + b] += torch.einsum("hgij,ihgd->jhd", w, do)
                dw = torch.einsum("ihgd,jhd->hgij", do, v[:b])
                dw = w * (dw - (dw * w).sum(-1, keepdim=True)) * scale
                dq[rows] = torch.einsum("hgij,jhd->ihgd", dw, k[:b]).flatten(1, 2)
                dk[at:at + b] += torch.einsum("hgij,ihgd->jhd", dw, q)
        at += n
    return {"o": o, "lse": lse} if case["way"] == "fwd" else {"dq": dq, "dk": dk, "dv": dv}


def _exact_paged(case, s):
    H, Hk, page, at = case["heads"], case["kv_heads"], case["page"], 0
    o = torch.zeros_like(s["q"])
    for b, (n, m) in enumerate(zip(s["lengths"], s["new"])):
        where = torch.arange(n, device=DEV)
        held, slot = s["tables"][b].long()[where // page], where % page
        k, v = s["k_pages"][held, slot], s["v_pages"][held, slot]
        for lo, hi in _exact_blocks(n, m, H):
            q = s["q"][at + lo:at + hi].unflatten(1, (Hk, H // Hk))
            w = torch.einsum("ihgd,jhd->hgij", q, k) * s["scale"]
            last = n - m + lo + torch.arange(hi - lo, device=DEV)
            w = torch.softmax(torch.where(where <= last[:, None], w, -math.inf), -1)
            o[at + lo:at + hi] = torch.einsum("hgij,jhd->ihgd", w, v).flatten(1, 2)
        at += m
    return {"o": o}


def _exact_cache(case, s):
    """Request by request and token by token, on the host."""
    page, tables, free = case["page"], s["tables"].tolist(), iter(s["free"].tolist())
    starts, positions, slots, taken = [0], [], [], 0
    for b, (n, m) in enumerate(zip(s["lengths"], s["new"])):
        for pos in range(n - m, n):
            if pos % page == 0:
                tables[b][pos // page] = next(free)
                taken += 1
            positions.append(pos)
            slots.append(tables[b][pos // page] * page + pos % page)
        starts.append(len(slots))
    at = torch.tensor(slots, device=DEV)
    pages = {}
    for n in ("k", "v"):
        flat = s[n + "_pages"].double().flatten(0, 1)
        flat[at] = s[n].double()
        pages[n + "_pages"] = flat.unflatten(0, (-1, page))
    return {"starts": _ints(starts), "lengths": _ints(s["lengths"]), "positions": _ints(positions), "slots": at,
            "taken": _ints([taken]), "tables": _ints(tables), **pages}
