"""Values, keys and queries that are not finite: only the rows that see them, and of a value only
its own dims, become what they make of it. The others are bit for bit what they are without."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


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


CASES = [
    # nh, nkv, d, ps, prefix, lens, new tokens
    (4, 4, 128, 64, 70, [50, 9], [8, 3]),                # drafted tokens, one row a token
    (8, 2, 64, 16, 0, [300, 129, 40], [4, 2, 1]),        # 16 rows over the end of a block
    (8, 2, 128, 32, 100, [700, 33], [16, 12]),           # 64 and 48 rows in tiles of 16
    (8, 2, 128, 64, 129, [200, 140], [30, 17]),          # 120 and 68 rows: one tile
    (8, 1, 64, 64, 0, [128, 260], [16, 13]),
    (8, 2, 128, 64, 300, [500, 65], [130, 65]),          # prompt chunks: tiles of two warpgroups
    (4, 1, 64, 32, 40, [900], [900]),                    # a whole prompt
    (3, 1, 128, 64, 0, [77], [77]),                      # groups that cross the tiles' rows
    (16, 1, 128, 16, 2000, [40, 300], [40, 9]),
    (2, 2, 64, 64, 0, [3], [7]),                         # more rows than keys
]


def setup(case):
    nh, nkv, d, ps, prefix, lens, news = CASES[case]
    pp, held = -(-prefix // ps), [-(-x // ps) for x in lens]
    pages = pp + sum(held)
    tables, at = torch.zeros(len(lens), max(held), dtype=torch.int32), pp
    for b, h in enumerate(held):
        tables[b, :h] = torch.arange(at, at + h)
        at += h
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    c = dict(q=normal(case, cu[-1], nh, d), k=normal(case + 50, pages, nkv, ps, d),
             v=normal(case + 90, pages, nkv, ps, d), cu=cu, tables=tables, d=d, ps=ps, pp=pp)

    def run(plan, **other):
        a = {**c, **other}
        out, lse = torch.full_like(c["q"], 7.0), torch.full((cu[-1], nh), 7.0, device="cuda")
        plan.attend(a["q"], ints(cu), ints(lens), tables.cuda(), a["k"], a["v"], out, lse=lse,
                    **(dict(prefix_table=ints(list(range(pp))), prefix_len=prefix) if prefix else {}))
        assert plan.status() == cfa_ok
        return out, lse

    cfa_ok = 0
    return c, run, lambda cfa: cfa.Paged(len(lens), cu[-1], nh, nkv, d, ps)


def places(case):
    """Own keys that some rows of their request see and others do not, the newest and an older one
    of each, and dims: (request, key, dim)."""
    _, _, d, _, _, lens, news = CASES[case]
    out = []
    for b, (L, n) in enumerate(zip(lens, news)):
        first = max(0, L - n + 1)
        for i, key in enumerate(sorted({L - 1, max(first, L - 2), (first + L) // 2, first})):
            if first <= key < L:
                out.append((b, key, (11 * i + 5 * b + 3) % d))
    return out


def rows_that_see(case, b, key):
    _, _, _, _, _, lens, news = CASES[case]
    return [sum(news[:b]) + i for i in range(news[b]) if key < max(0, lens[b] - news[b] + i + 1)]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_values_seen_by_some_rows(cfa, case, bad):
    c, run, plan_of = setup(case)
    G = c["q"].shape[1] // c["v"].shape[1]
    want_bad = torch.zeros(c["q"].shape, dtype=torch.bool, device="cuda")
    zero, spoiled = c["v"].clone(), c["v"].clone()
    for n, (b, key, dim) in enumerate(places(case)):
        g = n % c["v"].shape[1]
        page, off = int(c["tables"][b, key // c["ps"]]), key % c["ps"]
        zero[page, g, off, dim], spoiled[page, g, off, dim] = 0.0, bad
        for t in rows_that_see(case, b, key):
            want_bad[t, g * G:(g + 1) * G, dim] = True
    with plan_of(cfa) as plan:
        base, lse = run(plan, v=zero)
        got, lse2 = run(plan, v=spoiled)
        again, _ = run(plan, v=spoiled)
    assert torch.all(torch.isfinite(base)) and torch.equal(lse, lse2)
    assert torch.equal(got[~want_bad], base[~want_bad])
    hit = got[want_bad]
    assert hit.numel() > 0
    # a weight that passes out of 32 bits times an infinity may be NaN: none is that small here
    assert torch.all(torch.isnan(hit)) if math.isnan(bad) else torch.all(hit == bad)
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("case", [2, 3, 5, 6])
def test_infinities_of_both_signs(cfa, case):
    """Rows that see only one have it; those that see both have NaN."""
    c, run, plan_of = setup(case)
    _, _, _, ps, _, lens, news = CASES[case]
    first, last = lens[0] - news[0] + 1, lens[0] - 1
    v = c["v"].clone()
    for key, x in ((first, math.inf), (last, -math.inf)):
        v[int(c["tables"][0, key // ps]), :, key % ps, 6] = x
    with plan_of(cfa) as plan:
        out, _ = run(plan, v=v)
    x = out[:news[0], :, 6]
    assert torch.all(torch.isfinite(x[0])) and torch.all(x[1:news[0] - 1] == math.inf)
    assert torch.all(torch.isnan(x[news[0] - 1]))
    assert torch.all(torch.isfinite(out[:news[0], :, :6])) and torch.all(torch.isfinite(out[news[0]:]))


@pytest.mark.parametrize("case", range(len(CASES)))
def test_a_whole_row_of_nan(cfa, case):
    """The newest token's key and value, as an overflow upstream leaves them: its own rows are NaN,
    all earlier ones as ever."""
    c, run, plan_of = setup(case)
    _, _, _, ps, _, lens, news = CASES[case]
    k, v = c["k"].clone(), c["v"].clone()
    own = torch.zeros(c["q"].shape[0], dtype=torch.bool, device="cuda")
    for b, L in enumerate(lens):
        page, off = int(c["tables"][b, (L - 1) // ps]), (L - 1) % ps
        k[page, :, off] = v[page, :, off] = math.nan
        own[rows_that_see(case, b, L - 1)] = True
    with plan_of(cfa) as plan:
        base, lse = run(plan)
        got, lse2 = run(plan, k=k, v=v)
    assert torch.equal(got[~own], base[~own]) and torch.equal(lse[~own], lse2[~own])
    assert torch.all(torch.isnan(got[own])) and torch.all(torch.isnan(lse2[own]))


@pytest.mark.parametrize("case", range(len(CASES)))
def test_a_query_that_is_nan(cfa, case):
    c, run, plan_of = setup(case)
    q, T, nh = c["q"].clone(), *c["q"].shape[:2]
    spoiled = torch.zeros(T, nh, dtype=torch.bool, device="cuda")
    _, _, _, _, prefix, lens, news = CASES[case]
    for b in range(len(lens)):
        t = c["cu"][b + 1] - 1
        spoiled[t, t % nh] = True
    q[spoiled] = math.nan
    with plan_of(cfa) as plan:
        base, lse = run(plan)
        got, lse2 = run(plan, q=q)
    assert torch.equal(got[~spoiled], base[~spoiled]) and torch.equal(lse[~spoiled], lse2[~spoiled])
    assert torch.all(torch.isnan(got[spoiled])) and torch.all(torch.isnan(lse2[spoiled]))


@pytest.mark.parametrize("case", [0, 4, 5])
def test_a_recorded_call_meets_them_in_turn(cfa, case):
    """Replays of one graph, with values that are finite, are not, and are again."""
    nh, nkv, d, ps, prefix, lens, news = CASES[case]
    c, run, plan_of = setup(case)
    v = c["v"].clone()
    key, out = lens[0] - 1, torch.zeros_like(c["q"])
    page, off = int(c["tables"][0, key // ps]), key % ps
    a = (c["q"], ints(c["cu"]), ints(lens), c["tables"].cuda(), c["k"], v, out)
    kw = dict(prefix_table=ints(list(range(c["pp"]))), prefix_len=prefix) if prefix else {}
    with plan_of(cfa) as plan:
        zero = c["v"].clone()
        zero[page, :, off, 9] = 0.0
        base, _ = run(plan, v=zero)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            plan.attend(*a, **kw)
        for x in (0.0, math.inf, 0.0, math.nan, -math.inf, -math.inf, 0.0):
            v[page, :, off, 9] = x
            g.replay()
            want = base.clone()
            if x != 0.0:
                want[rows_that_see(case, 0, key), :, 9] = x
            assert torch.equal(torch.nan_to_num(out, nan=5.0), torch.nan_to_num(want, nan=5.0))
        assert plan.status() == cfa.CFA_OK


def test_many_rows_meet_them(cfa):
    """A long prompt: the pass behind the call is one load a token, not one a pair of tokens."""
    nh, nkv, d, ps, n = 8, 2, 128, 64, 20000
    pages = -(-n // ps)
    q, k, v = normal(1, n, nh, d), normal(2, pages, nkv, ps, d), normal(3, pages, nkv, ps, d)
    out, tables = torch.empty_like(q), ints([list(range(pages))])
    key = 12345
    v[key // ps, 1, key % ps, 100] = math.inf
    with cfa.Paged(1, n, nh, nkv, d, ps) as plan:
        plan.attend(q, ints([0, n]), ints([n]), tables, k, v, out)
        assert plan.status() == cfa.CFA_OK
    want = torch.zeros(n, nh, d, dtype=torch.bool, device="cuda")
    want[key:, 4:, 100] = True
    assert torch.equal(~torch.isfinite(out), want) and torch.all(out[want] == math.inf)
