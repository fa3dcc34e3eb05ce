"""Paged attention's errors as a whole, and caches value by value.

The bound on the relative L2 error of a row (a token's head) against 64 bits, for values that
are independent with mean zero. A rounding to bf16 is off by at most 2^-8 of the value, evenly
spread, so by 2^-8 / sqrt(3) = 0.00226 in the root mean square at most (where every number lies
at the lower end of its binade). The result is rounded once. Each weight is rounded once too:
with independent values the sum of the errors delta_j w_j v_j has the size of delta times the
sum of the w_j v_j itself, again 0.00226. Together at most 0.0032 over many rows; a single row
of 64 dims or more gets twice that. A value that is left out, of some n with weights like these,
changes its row by about 1 / sqrt(n): 0.018 at 3000 keys."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

ALL, ROW = 0.0032, 0.0064


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


def batch(seed, nh, nkv, d, ps, prefix, lens, news):
    g = torch.Generator().manual_seed(seed)
    held, pp = [-(-x // ps) for x in lens], -(-prefix // ps)
    ids = torch.randperm(pp + sum(held) + 1, generator=g).tolist()
    tables, at = torch.zeros(len(lens), max(held), dtype=torch.int32), pp
    for b, h in enumerate(held):
        tables[b, :h] = torch.tensor(ids[at:at + h], dtype=torch.int32)
        at += h
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    return dict(q=normal(seed, cu[-1], nh, d), kp=normal(seed + 1, len(ids), nkv, ps, d),
                vp=normal(seed + 2, len(ids), nkv, ps, d), tables=tables.cuda(), cu=cu, lens=lens,
                prefix_table=ids[:pp], prefix=prefix)


def exact(c, leave_out=False):
    """In 64 bits; leave_out: without the value of every row's middle key."""
    (T, nh, d), nkv = c["q"].shape, c["kp"].shape[1]
    G, out = nh // nkv, torch.empty(c["q"].shape, dtype=torch.float64, device="cuda")

    def rows(pages, table, n, g):
        return pages[table.long(), g].reshape(-1, d)[:n].double()

    pt = ints(c["prefix_table"])
    for g in range(nkv):
        for b, L in enumerate(c["lens"]):
            t0, t1 = c["cu"][b], c["cu"][b + 1]
            K, V = (torch.cat((rows(x, pt, c["prefix"], g), rows(x, c["tables"][b], L, g)))
                    for x in (c["kp"], c["vp"]))
            s = torch.einsum("tgd,kd->tgk", c["q"][t0:t1, g * G:(g + 1) * G].double(), K) / math.sqrt(d)
            last = c["prefix"] + L - (t1 - t0) + torch.arange(t1 - t0, device="cuda")
            s.masked_fill_(torch.arange(len(K), device="cuda") > last[:, None, None], -math.inf)
            w = torch.softmax(s, -1)
            if leave_out:
                w[torch.arange(t1 - t0), :, last // 2] = 0
            out[t0:t1, g * G:(g + 1) * G] = w @ V
    return out


CASES = [
    # nh, nkv, d, ps, prefix, lens, new tokens
    (8, 8, 128, 64, 700, [900, 400, 55], [1, 1, 1]),          # one row a key head
    (32, 8, 128, 16, 1000, [300, 900, 31, 600] * 5, [1] * 20),  # 80 rows over the prefix
    (64, 8, 64, 64, 0, [1500, 2000, 80], [1, 1, 1]),          # without a prefix
    (8, 2, 128, 32, 1234, [700] * 12, [8, 3, 5, 1] * 3),      # drafted tokens, 16-row tiles
    (16, 2, 64, 64, 513, [700, 900], [9, 15]),                # 72 and 120 rows of their own
    (8, 2, 128, 64, 600, [1500, 700], [300, 129]),            # prompt chunks
    (8, 2, 64, 128, 0, [900, 1300], [900, 200]),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_error_as_a_whole(cfa, case):
    nh, nkv, d, ps, prefix, lens, news = CASES[case]
    c = batch(40 + 10 * case, nh, nkv, d, ps, prefix, lens, news)
    out = torch.empty_like(c["q"])
    kw = dict(prefix_table=ints(c["prefix_table"]), prefix_len=prefix) if prefix else {}
    with cfa.Paged(len(lens), sum(news), nh, nkv, d, ps) as plan:
        plan.attend(c["q"], ints(c["cu"]), ints(lens), c["tables"], c["kp"], c["vp"], out, **kw)
        assert plan.status() == cfa.CFA_OK
    want = exact(c)

    def off(x):
        e, n = (x - want).norm(dim=-1), want.norm(dim=-1)
        return float(e.norm() / n.norm()), float((e / n).max())

    whole, worst = off(out.double())
    assert whole <= ALL and worst <= ROW, (whole, worst)
    # the bounds see one value of each row that is left out
    whole, worst = off(exact(c, leave_out=True))
    assert whole > 2 * ALL and worst > ROW


@pytest.mark.parametrize("nh,nkv,d,ps", [(8, 2, 128, 16), (4, 4, 64, 64)])
def test_values_of_several_layers_and_steps(cfa, nh, nkv, d, ps):
    """Tables, then layers that append: the value caches are copies bit for bit, and what no slot
    names stays as it was, in the key caches too."""
    B, T, pages = 4, 16, 40
    caches = [(normal(i, pages, nkv, ps, d), normal(9 + i, pages, nkv, ps, d)) for i in range(2)]
    model = [(k.clone(), v.clone()) for k, v in caches]
    lens, fresh, pool = ints([0, 5, 15, 31]), ints([0] * B), ints([3, pages - 8])
    tables = torch.full((B, 6), -1, dtype=torch.int32, device="cuda")
    tables[1:, :2] = ints([[pages - 1, pages - 2], [pages - 3, pages - 4], [pages - 5, pages - 6]])
    free, cu, pos, slots = ints(range(pages - 8)), ints([0] * (B + 1)), ints([0] * T), ints([0] * T)
    turned, out = (torch.zeros(T, nh, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    with cfa.Paged(B, T, nh, nkv, d, ps) as plan:
        plan.set_rope()
        for step, new in enumerate(([1, 1, 1, 1], [3, 0, 5, 2], [0, 8, 1, 7])):
            fresh.copy_(ints(new))
            plan.build_tables(lens, fresh, free, pool, tables, lens, pool, cu, pos, slots, base=3)
            where = slots.tolist()[:sum(new)]
            assert slots.tolist()[sum(new):] == [-1] * (T - sum(new))
            for i, ((kp, vp), (mk, mv)) in enumerate(zip(caches, model)):
                q, k, v = normal(50 + step, T, nh, d), normal(60 + i, T, nkv, d), normal(70 + step + i, T, nkv, d)
                plan.layer(q, k, v, pos, slots, cu, lens, tables, kp, vp, turned, out)
                assert plan.status() == cfa.CFA_OK
                for t, s in enumerate(where):
                    mv[s // ps, :, s % ps] = v[t]
                    mk[s // ps, :, s % ps] = kp[s // ps, :, s % ps]
                assert torch.equal(vp, mv) and torch.equal(kp, mk)
    assert lens.tolist() == [4, 14, 22, 41]


def test_tables_into_other_counters(cfa):
    """pool_out and lens_out apart from pool and lens, which stay as they were."""
    lens, pool, x, y = ints([15, 16, 0, 7]), ints([1, 6]), ints([-9] * 4), ints([-9] * 4)
    tables = ints([[9, -1, -1]] * 4)
    cu, pos, slots = ints([0] * 5), ints([0] * 8), ints([0] * 8)
    with cfa.Paged(4, 8, 8, 2, 64, 16) as plan:
        plan.build_tables(lens, ints([2, 1, 0, 1]), ints(range(20, 26)), pool, tables, y, x[:2], cu, pos, slots)
        assert plan.status() == cfa.CFA_OK
    assert x.tolist() == [3, 6, -9, -9] and pool.tolist() == [1, 6]
    assert y.tolist() == [17, 17, 0, 8] and lens.tolist() == [15, 16, 0, 7]
    assert cu.tolist() == [0, 2, 3, 3, 4] and tables.tolist() == [[9, 21, -1], [9, 22, -1], [9, -1, -1], [9, -1, -1]]
    assert slots.tolist() == [9 * 16 + 15, 21 * 16, 22 * 16, 9 * 16 + 7, -1, -1, -1, -1]
