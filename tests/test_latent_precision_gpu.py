"""The error of latent attention as a whole, against 64 bits: no more than what the two roundings to bf16
that it is allowed, the weights' and the result's, come to.

A rounding to bf16 is off by at most 2^-8 of the value; spread evenly, by 2^-8 / sqrt(3) of it in the mean square
(less, as few values lie just above a power of two: 0.74 of that for values spread over their logarithm). The
weights' roundings do not depend on one another, so a result sum_j w_j v_j / l is off by 2^-8 / sqrt(3) times
r = sqrt(sum_j w_j^2 v_j^2) / l in the mean square, and its own rounding by that times the result y:
  sum err^2 <= 2^-16 / 3 (sum r^2 + sum y^2).
Sums in fp32 (some 2^-20 of the result) are far below. What is left to chance is small over the 10^5 results of
a case, and 0.74 leaves a third for it. Weights with one bit less would come to 1.16 of the bound.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ROW, QK, C, V = 576, 192, 512, 128


@pytest.fixture(scope="module")
def cfa():
    from out_proj_block_gb300 import build
    build.build()
    from out_proj_block_gb300 import cfa
    return cfa


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def normal(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def offsets(counts):
    return [0, *np.cumsum(counts).tolist()]


class Sums:
    """Squares of the errors, and what they may come to."""

    def __init__(self):
        self.err = self.may = 0.0

    def add(self, got, w, v):
        """Weights w [tokens, keys], 0 where a token does not see a key, and values v [keys, dims]."""
        l = w.sum(1, keepdim=True)
        y, r2 = w @ v / l, w.square() @ v.square() / l.square()
        self.err += (got.double() - y).square().sum().item()
        self.may += 2.0 ** -16 / 3.0 * (r2.sum() + y.square().sum()).item()

    def check(self):
        assert self.err <= self.may, f"{math.sqrt(self.err / self.may):.3f} of what the roundings come to"


def weights_of(s, n, L):
    """exp of scores [n, L] less their maximum, for the last n of L tokens."""
    see = torch.arange(L, device="cuda") <= torch.arange(L - n, L, device="cuda")[:, None]
    s = s.masked_fill(~see, -math.inf)
    return torch.exp(s - s.amax(1, keepdim=True))


@pytest.mark.parametrize("H,ps,pairs", [
    (128, 64, [(1, 20000)]),                                       # one request over the whole GPU
    (32, 64, [(1, 9000), (2, 3100), (1, 500)]),                    # cut tiles, whole tiles
    (20, 128, [(1 + i % 4, 700 + 331 * i) for i in range(12)]),    # drafted tokens
    (128, 16, [(1, 1500 + 17 * i) for i in range(30)]),
])
def test_attend(cfa, H, ps, pairs):
    B, cu = len(pairs), offsets([n for n, _ in pairs])
    held = [-(-L // ps) for _, L in pairs]
    ids = np.random.default_rng(H).permutation(sum(held))
    tables = torch.zeros(B, max(held), dtype=torch.int32)
    for b, at in enumerate(offsets(held)[:-1]):
        tables[b, :held[b]] = torch.from_numpy(ids[at:at + held[b]].astype(np.int32))
    q, pages = normal(1, cu[-1], H, ROW), normal(2, sum(held), ps, ROW)
    out = torch.empty(cu[-1], H, C, dtype=torch.bfloat16, device="cuda")
    with cfa.Latent(B, cu[-1], H, ps) as plan:
        plan.attend(q, ints(cu), ints([L for _, L in pairs]), tables.cuda(), pages, out)
        assert plan.status() == cfa.CFA_OK
    sums = Sums()
    for b, (n, L) in enumerate(pairs):
        rows = pages[tables[b, :held[b]].long().cuda()].flatten(0, 1)[:L].double()
        for h in range(H):
            s = q[cu[b]:cu[b + 1], h].double() @ rows.T / math.sqrt(QK)
            sums.add(out[cu[b]:cu[b + 1], h], weights_of(s, n, L), rows[:, :C])
    sums.check()


@pytest.mark.parametrize("H,pairs", [
    (2, [(2500, 2500)]),                                           # tasks split along the keys
    (16, [(600, 4000), (700, 2900)]),                              # two tiles in a row of a head in a task
    (20, [(300, 300 + 97 * i) for i in range(8)]),
    (32, [(1000, 1500), (763, 763)]),
])
def test_expanded(cfa, H, pairs):
    B, cu, ck = len(pairs), offsets([n for n, _ in pairs]), offsets([L for _, L in pairs])
    q, kv, k_rope = normal(1, cu[-1], H, QK), normal(2, ck[-1], H, 256), normal(3, ck[-1], 64)
    out = torch.empty(cu[-1], H, V, dtype=torch.bfloat16, device="cuda")
    with cfa.Latent(B, cu[-1], H, 64) as plan:
        plan.attend_expanded(q, kv, k_rope, ints(cu), ints(ck), out)
        assert plan.status() == cfa.CFA_OK
    sums = Sums()
    for b, (n, L) in enumerate(pairs):
        keys = slice(ck[b], ck[b + 1])
        for h in range(H):
            k = torch.cat((kv[keys, h, :128], k_rope[keys]), 1).double()
            s = q[cu[b]:cu[b + 1], h].double() @ k.T / math.sqrt(QK)
            sums.add(out[cu[b]:cu[b + 1], h], weights_of(s, n, L), kv[keys, h, 128:].double())
    sums.check()
