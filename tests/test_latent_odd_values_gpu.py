"""Values that are not finite in the expanded form of latent attention: they stay with the tokens that see
them, however the call is cut, and do not hold up the rest of a batch."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

QK, V = 192, 128
BAD = (float("inf"), float("-inf"), float("nan"))


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


class Call:
    """pairs: (new tokens, keys) of each request."""

    def __init__(self, cfa, H, pairs, seed=1, lead=1):
        self.pairs, self.H = pairs, H
        self.cu, self.ck = [lead], [0]
        for n, L in pairs:
            self.cu.append(self.cu[-1] + n)
            self.ck.append(self.ck[-1] + L)
        self.T, S = self.cu[-1] + 1, max(1, self.ck[-1])
        self.q, self.kv, self.k_rope = normal(seed, self.T, H, QK), normal(seed + 1, S, H, 256), normal(seed + 2, S, 64)
        self.cu_d, self.ck_d = ints(self.cu), ints(self.ck)
        self.plan = cfa.Latent(len(pairs), self.T, H, 64)
        self.out = torch.empty(self.T, H, V, dtype=torch.bfloat16, device="cuda")

    def run(self):
        self.plan.attend_expanded(self.q, self.kv, self.k_rope, self.cu_d, self.ck_d, self.out)
        return self.out

    def fresh(self):
        self.out.fill_(5.0)
        return self.run().clone()

    def poison(self, rng, count):
        """Bad values, most of them among the keys that only some tokens see; and what the tokens that see them
        are to show: the sum of what they see, 0 where that is nothing."""
        want = torch.zeros(self.T, self.H, V, dtype=torch.float32, device="cuda")
        held = [b for b, (n, L) in enumerate(self.pairs) if n and L]
        for _ in range(count):
            b = held[int(rng.integers(len(held)))]
            n, L = self.pairs[b]
            j = int(rng.integers(max(0, L - n), L)) if rng.random() < 0.8 else int(rng.integers(L))
            h, d, bad = int(rng.integers(self.H)), int(rng.integers(V)), BAD[int(rng.integers(3))]
            self.kv[self.ck[b] + j, h, 128 + d] = bad
        for b in held:
            n, L = self.pairs[b]
            v = self.kv[self.ck[b]:self.ck[b + 1], :, 128:].float()
            seen = torch.cumsum(torch.where(v.isfinite(), 0.0, v), 0)  # what keys up to j hold
            see = torch.arange(L - n, L, device="cuda")                 # the last key that each token sees
            some = see >= 0
            want[self.cu[b]:self.cu[b + 1]][some] = seen[see[some]]
        return want


SHAPES = [
    (1, [(2500, 2500)]),                                  # tasks that are split along the keys
    (3, [(600, 3000), (257, 2700), (800, 2900)]),         # two tiles in a row of a head in a task
    (7, [(130, 2100), (257, 257), (1, 3000), (300, 150)]),
    (20, [(512 - n, 100 + n) for n in range(40)]),        # tokens that see no key
    (3, [(n % 5, n % 7) for n in range(1024)]),           # the most requests, some without tokens or keys
    (5, [(33, 33)] * 30),
    (32, [(1500, 1500), (1035, 1035), (763, 900)]),
    (128, [(520, 3000)]),
    (1, [(1, 2700), (513, 2561), (1, 1)]),                # (an odd number of heads beside a request of one token)
]


@pytest.mark.parametrize("H,pairs", SHAPES)
@pytest.mark.parametrize("count", [1, 40])
def test_bad_values_stay_with_their_tokens(cfa, H, pairs, count):
    rng = np.random.default_rng(H + count)
    c = Call(cfa, H, pairs)
    good, kv = c.fresh(), c.kv.clone()
    for _ in range(6 if count == 1 else 2):
        want = c.poison(rng, count)
        got = c.fresh()
        clean = want == 0
        assert torch.equal(got.view(torch.int16)[clean], good.view(torch.int16)[clean])
        x, y = got[~clean].float(), want[~clean]
        assert torch.equal(x.isnan(), y.isnan()) and torch.equal(x[~x.isnan()], y[~y.isnan()])
        c.kv.copy_(kv)
        assert torch.equal(c.fresh().view(torch.int16), good.view(torch.int16))  # nothing is left for the next call
    assert c.plan.status() == cfa.CFA_OK


def test_bad_values_in_recorded_calls(cfa):
    """Bad values that come and go between replays."""
    c = Call(cfa, 5, [(300, 900), (65, 65), (2000, 2700)])
    good, kv = c.fresh(), c.kv.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    rng = np.random.default_rng(3)
    for _ in range(4):
        want = c.poison(rng, 10)
        graph.replay()
        clean = want == 0
        assert torch.equal(c.out.view(torch.int16)[clean], good.view(torch.int16)[clean])
        assert not c.out[~clean].isfinite().any()
        c.kv.copy_(kv)
        graph.replay()
        assert torch.equal(c.out.view(torch.int16), good.view(torch.int16))
    assert c.plan.status() == cfa.CFA_OK


@pytest.mark.parametrize("H,pairs", [(32, [(1500, 1500), (1035, 1035), (1447, 1447), (1135, 1135), (763, 763)]),
                                     (32, [(100, 100)] * 64)])
def test_one_bad_value_does_not_hold_up_its_batch(cfa, H, pairs):
    """What is added is a part of the keys' bytes: less than the attention's own time (twice is allowed for it)."""
    c = Call(cfa, H, pairs)

    def fastest():
        times = []
        for _ in range(8):
            begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            begin.record()
            for _ in range(4):
                c.run()
            end.record()
            torch.cuda.synchronize()
            times.append(begin.elapsed_time(end))
        return min(times)

    fastest()
    clean = fastest()
    c.kv[c.ck[1] - 30, H // 2, 128 + 7] = float("inf")
    assert fastest() < 3.0 * clean
    assert c.plan.status() == cfa.CFA_OK
