"""An HMM whose transition copies are steered by a sequence model.

The circuit's LowRank factors FA[t], FB[t] (``hmm_lowrank_fwd_bwd``) are made by a small
network from the tokens up to position t: embedding, layer norm, linear attention with a
decay for each head, layer norm, two linear heads. Training follows the circuit's gradients
dFA, dFB back through the network, updates its matrices by orthogonalised steps and the
circuit's own tables by the EM M-step; serving makes the factors one position at a time
from the attention's states.

    python examples/factor_network.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import log_space_sum_gb300 as pc  # noqa: E402


class FactorNetwork:
    """Tokens [B,T] -> factors FA [T-1,B,H,K], FB [T-1,B,K,H]; ``dtype`` is that of the
    activations (the weights are float32)."""

    def __init__(self, vocab, latents, rank, width=64, heads=2, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, std: std * torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.H, self.K, self.D, self.h, self.dtype = latents, rank, width, heads, dtype
        self.p = dict(emb=r(vocab, width, std=1.0), qkv=r(width, 3 * width, std=width ** -0.5),
                      out=r(width, width, std=width ** -0.5),
                      fa=r(width, latents * rank, std=0.3 * width ** -0.5),
                      fb=r(width, rank * latents, std=0.3 * width ** -0.5))
        self.norms = [[torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")] for _ in range(2)]
        self.log_decay = -torch.exp2(-1.0 - torch.arange(heads, device="cuda"))  # memories of a few tokens
        self.scale = (width // heads) ** -0.5

    def _mm(self, x, name):
        return x @ self.p[name].to(x.dtype)

    def _heads(self, x):
        return x.unflatten(-1, (self.h, self.D // self.h))

    def _factors(self, z):
        """[B,T,D] -> FA [T,B,H,K], FB [T,B,K,H] in float32, as the circuit takes them."""
        fa = self._mm(z, "fa").unflatten(-1, (self.H, self.K))
        fb = self._mm(z, "fb").unflatten(-1, (self.K, self.H))
        return fa.transpose(0, 1).float().contiguous(), fb.transpose(0, 1).float().contiguous()

    def forward(self, tokens):
        """Factors for every copy, and what the backward reads."""
        t = tokens[:, :-1].long()
        e = self.p["emb"][t].to(self.dtype)
        z1, m1, r1 = pc.layer_norm_fwd(e, *self.norms[0])
        qkv = self._mm(z1, "qkv")
        q, k, v = (self._heads(x) for x in qkv.split(self.D, -1))  # slices, not copies
        o, _ = pc.linear_attention_fwd(q, k, v, self.log_decay, scale=self.scale)
        x = e + self._mm(o.flatten(2), "out")
        z2, m2, r2 = pc.layer_norm_fwd(x, *self.norms[1])
        return self._factors(z2), (t, e, z1, m1, r1, q, k, v, o, x, z2, m2, r2)

    def backward(self, saved, dFA, dFB):
        """Gradients of the parameters from the circuit's dFA, dFB."""
        t, e, z1, m1, r1, q, k, v, o, x, z2, m2, r2 = saved
        g = {}

        def linear(inp, dout, name):
            g[name] = inp.flatten(0, 1).t().float() @ dout.flatten(0, 1).float()
            return dout @ self.p[name].to(dout.dtype).t()

        da = dFA.transpose(0, 1).flatten(2).to(self.dtype)
        db = dFB.transpose(0, 1).flatten(2).to(self.dtype)
        dz2 = linear(z2, da, "fa") + linear(z2, db, "fb")
        dx, g["w2"], g["b2"] = pc.layer_norm_bwd(dz2, x, self.norms[1][0], m2, r2)
        do = self._heads(linear(o.flatten(2), dx, "out"))
        dqkv = torch.empty(*z1.shape[:2], 3 * self.D, dtype=self.dtype, device="cuda")
        parts = [self._heads(s) for s in dqkv.split(self.D, -1)]
        pc.linear_attention_bwd(q, k, v, self.log_decay, do, scale=self.scale, dq=parts[0], dk=parts[1], dv=parts[2])
        de, g["w1"], g["b1"] = pc.layer_norm_bwd(linear(z1, dqkv, "qkv"), e, self.norms[0][0], m1, r1)
        g["emb"] = torch.zeros_like(self.p["emb"]).index_add_(0, t.flatten(), (de + dx).flatten(0, 1).float())
        return g

    def update(self, g, lr):
        """Ascent: matrices by their orthogonalised gradients, the rest by a scaled one."""
        for name in ("qkv", "out", "fa", "fb"):
            step = pc.orthogonalize(g[name].to(torch.bfloat16))
            self.p[name] += lr * step.float()
        for t, n in ((self.p["emb"], "emb"), (self.norms[0][0], "w1"), (self.norms[0][1], "b1"),
                     (self.norms[1][0], "w2"), (self.norms[1][1], "b2")):
            t += lr * g[n] / g[n].norm().clamp(min=1e-12) * t.numel() ** 0.5 * 0.1

    def start(self, batch):
        """States for serving: one position at a time."""
        d = self.D // self.h
        return torch.zeros(batch, self.h, d, d, device="cuda")

    def step(self, tokens, state):
        """The factors after one more token each (tokens [B]); the state is advanced."""
        e = self.p["emb"][tokens.long()].to(self.dtype)
        z1, _, _ = pc.layer_norm_fwd(e, *self.norms[0])
        q, k, v = (self._heads(x) for x in self._mm(z1, "qkv").split(self.D, -1))
        o = pc.linear_attention_step(q, k, v, self.log_decay, state, scale=self.scale)
        z2, _, _ = pc.layer_norm_fwd(e + self._mm(o.flatten(1), "out"), *self.norms[1])
        fa, fb = self._factors(z2[:, None])
        return fa[0], fb[0]


def train_step(net, circuit, tokens, lr, precision="auto"):
    """One step on a batch: returns the mean log-likelihood before it."""
    (FA, FB), saved = net.forward(tokens)
    r = pc.hmm_lowrank_fwd_bwd(tokens, circuit["pi"], circuit["A"], circuit["E"], FA, FB, precision=precision)
    net.update(net.backward(saved, r["dFA"], r["dFB"]), lr)
    pc.em_normalize(r["dA"], circuit["A"], r["W"])  # the conditional M-step of the tied transitions
    pc.em_normalize(r["dE"] + 1e-3, circuit["E"])
    pc.em_normalize(r["dpi"] + 1e-3, circuit["pi"])
    return r["ll"].mean().item()


def toy(batch, length, vocab, seed):
    """Sequences in which each token follows from the one before the last, mostly."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(0, vocab, (batch, length), generator=g)
    for t in range(2, length):
        keep = torch.rand(batch, generator=g) < 0.9
        x[:, t] = torch.where(keep, (x[:, t - 2] * 5 + 1) % vocab, x[:, t])
    return x.to(torch.int32).cuda()


def make_circuit(vocab, latents, seed):
    g = torch.Generator().manual_seed(seed)
    rows = lambda *s: torch.softmax(torch.randn(*s, generator=g), -1).cuda()  # noqa: E731
    return dict(pi=rows(latents), A=rows(latents, latents), E=rows(latents, vocab))


def main(steps=40, batch=64, length=24, vocab=24, latents=64, rank=4):
    net, circuit = FactorNetwork(vocab, latents, rank), make_circuit(vocab, latents, 1)
    lls = []
    for i in range(steps):
        lls.append(train_step(net, circuit, toy(batch, length, vocab, 100 + i), lr=0.05))
        if i % 10 == 0 or i + 1 == steps:
            print(f"step {i}: mean log-likelihood {lls[-1]:.3f}")
    # serving: the same factors, a position at a time
    tokens = toy(4, length, vocab, 7)
    (FA, FB), _ = net.forward(tokens)
    state, off = net.start(4), 0.0
    for t in range(length - 1):
        fa, fb = net.step(tokens[:, t], state)
        off = max(off, (fa - FA[t]).abs().max().item(), (fb - FB[t]).abs().max().item())
    print(f"served factors differ from the prompt's by {off:.4f} at most (bf16 activations)")
    pc.device_status()
    return lls, off


if __name__ == "__main__":
    main()
