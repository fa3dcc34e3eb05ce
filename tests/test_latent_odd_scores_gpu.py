"""Scores that are not finite in latent attention over expanded keys, and infinite values whose weight is 0: what
the tokens that see them show, and that no others do."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

QK, V = 192, 128


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


def run(cfa, q, kv, k_rope, cu, ck, scale=None):
    T, H = q.shape[:2]
    out, lse = torch.empty(T, H, V, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, device="cuda")
    with cfa.Latent(len(cu) - 1, T, H, 64) as plan:
        plan.attend_expanded(q, kv, k_rope, ints(cu), ints(ck), out, scale=scale, lse=lse)
        assert plan.status() == cfa.CFA_OK
    return out, lse


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["key", "rope"])
@pytest.mark.parametrize("n,L,j", [(200, 300, 250), (200, 300, 20), (600, 2900, 2500), (600, 2900, 2750), (1, 700, 699),
                                   (2500, 2500, 1200)])
def test_scores_show_where_they_are_seen(cfa, bad, where, n, L, j):
    """NaN or +inf: the token's head is NaN. -inf: the key has weight 0."""
    H, h = 3, 1
    q, kv, k_rope = normal(1, n + 40, H, QK), normal(2, L + 40, H, 256), normal(3, L + 40, 64)
    cu, ck = [0, n, n + 40], [0, L, L + 40]
    good, gl = run(cfa, q, kv, k_rope, cu, ck)
    if where == "key":
        kv[j, h, 5] = bad
        score = torch.full((n + 40, H), 1.0, device="cuda")
        score[:, h] = q[:, h, 5].float() * bad
    else:
        k_rope[j, 9] = bad
        score = q[:, :, 128 + 9].float() * bad
    out, lse = run(cfa, q, kv, k_rope, cu, ck)
    first = max(0, n - L + j)  # the first token that sees the key
    sees = torch.zeros(n + 40, 1, dtype=torch.bool, device="cuda")
    sees[first:n] = True
    hit = sees & (score.isnan() | (score == math.inf))
    none = sees & (score == -math.inf)
    assert same(out[~hit & ~none], good[~hit & ~none]) and torch.equal(lse[~hit & ~none], gl[~hit & ~none])
    assert out[hit].isnan().all() and lse[hit].isnan().all()
    assert hit.any() or none.any()
    # without that key, in 64 bits: lse as ever to 1e-4, results to 2^-8 of the weights' and the result's rounding
    rows = none.nonzero()
    for t, g in rows[:: max(1, len(rows) // 8)].tolist():
        see = [k for k in range(L - n + t + 1) if k != j]
        k = torch.cat((kv[see, g, :128], k_rope[see]), 1).double()
        s, v = k @ q[t, g].double() / math.sqrt(QK), kv[see, g, 128:].double()
        if not see:
            assert not out[t, g].any() and lse[t, g] == -math.inf
            continue
        w = torch.softmax(s, 0)
        y, size = w @ v, w @ v.abs()
        assert torch.all((out[t, g].double() - y).abs() <= 2.0 ** -8 * (1.0625 * size + y.abs()))
        assert abs(lse[t, g].item() - torch.logsumexp(s, 0).item()) <= 1e-4


def test_scores_of_minus_infinity_only(cfa):
    """A token's head that has no other scores is as one that sees nothing."""
    q, kv, k_rope = normal(1, 3, 2, QK).abs(), normal(2, 3, 2, 256), normal(3, 3, 64)
    kv[:2, 0, 7] = float("-inf")
    out, lse = run(cfa, q, kv, k_rope, [0, 3], [0, 3])
    assert not out[:2, 0].any() and torch.all(lse[:2, 0] == -math.inf)
    assert out.isfinite().all() and lse[2].isfinite().all() and lse[:, 1].isfinite().all()


@pytest.mark.parametrize("n,L,j", [(200, 300, 250), (200, 300, 20), (1000, 1000, 400)])
def test_infinite_values_of_weight_zero(cfa, n, L, j):
    """Infinity or NaN, in that dim of the tokens that see it."""
    H = 2
    q, kv, k_rope = normal(1, n, H, QK), normal(2, L, H, 256), normal(3, L, 64)
    q[:, :, 0], kv[:, :, 0], kv[j, :, 0] = 16.0, 8.0, -64.0  # a score some 1150 * scale below the others
    good, _ = run(cfa, q, kv, k_rope, [0, n], [0, L], scale=1.0)
    kv[j, 1, 128 + 3] = float("inf")
    out, _ = run(cfa, q, kv, k_rope, [0, n], [0, L], scale=1.0)
    first = max(0, n - L + j)
    assert not out[first:, 1, 3].isfinite().any()
    out[first:, 1, 3] = good[first:, 1, 3]
    assert same(out, good)
