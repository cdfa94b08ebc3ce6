"""The barriers between the state warps, the issuer and the tensor pipe in the launch that
leaves the segments' states (linear_attention_tc.cuh), as a model: parity barriers, one warp
delayed at will. A warp announces the operands of chunk n + 1 before it waits for the products of
chunk n, so these products' barrier must not be reused by chunk n + 1."""
import random

import pytest

WARPS, CHUNKS = 8, 12


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def passed(self, parity):  # as mbarrier.try_wait.parity
        return (self.phase & 1) != parity


def runs_through(barriers, seed):
    rng = random.Random(seed)
    ready, free, d_free = ([Barrier(n) for _ in range(2)] for n in (WARPS, 1, WARPS))
    d_full = [Barrier(1) for _ in range(barriers)]
    pipe = []  # what the issuer has committed, in order

    def products(n):
        return d_full[n % barriers], n // barriers & 1

    def announce(n):
        for group in (0, 1):
            yield "wait", free[group], n & 1 ^ 1
            yield "arrive", ready[group]

    def state_warp():
        for n in range(CHUNKS):
            if n == 0:
                yield from announce(0)
            if n + 1 < CHUNKS:
                yield from announce(n + 1)
            yield ("wait", *products(n))
            yield "arrive", d_free[n & 1]

    def issuer():
        for n in range(CHUNKS):
            yield "wait", d_free[n & 1], n >> 1 & 1 ^ 1
            for group in (0, 1):
                yield "wait", ready[group], n & 1
                yield "commit", free[group]
            yield "commit", products(n)[0]

    roles = [state_warp() for _ in range(WARPS)] + [issuer()]
    at, slow = [next(r) for r in roles], rng.randrange(WARPS)
    while any(a is not None for a in at):
        can = [i for i, a in enumerate(at) if a is not None and (a[0] != "wait" or a[1].passed(a[2]))]
        can += ["pipe"] if pipe else []
        if not can:
            return False
        quick = [i for i in can if i != slow] or can
        i = rng.choice(quick if rng.random() < 0.97 else can)
        if i == "pipe":
            pipe.pop(0).arrive()
            continue
        if at[i][0] == "arrive":
            at[i][1].arrive()
        elif at[i][0] == "commit":
            pipe.append(at[i][1])
        at[i] = next(roles[i], None)
    return True


@pytest.mark.parametrize("barriers,stuck", [(1, True), (2, False)])
def test_a_delayed_warp(barriers, stuck):
    assert any(not runs_through(barriers, seed) for seed in range(200)) == stuck
