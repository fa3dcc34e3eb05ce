"""Paged-cache operators on the GPU against their fp64 definitions.

Tolerances, from the roundings alone (a bf16 rounding is at most 2^-8 of the value):
  append     one rounding of y: 2^-8 |y|; the angle and the sine in fp32 are within
             1e-6 of the pair's magnitude.
  attention  the weights are rounded to bf16 for their product with v (2^-8 each, so at
             most 2^-8 sum w|v| / sum w), the result once more (2^-8 |o|); fp32 sums,
             scores and exponentials add under a sixteenth of that. lse: scores of magnitude
             s sum d products in fp32, within d 2^-24 sum |q k| scale, below 1e-4 here.
"""
import math

import numpy as np
import pytest
import torch

from oracle import cfa_oracle_paged as ref

pytestmark = pytest.mark.gpu

H8 = 2.0 ** -8


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


def f64(t):
    return t.detach().double().cpu().numpy()


# --------------------------------------------------------------------- tables


def tables_case(B, ps, seed, most_cached=300, most_fresh=3, spare=5, pad=3):
    r = np.random.default_rng(seed)
    lens = [int(v) for v in r.integers(0, most_cached + 1, B)]
    fresh = [int(v) for v in r.integers(0, most_fresh + 1, B)]
    if sum(fresh) == 0:
        fresh[0] = 1
    width = max(-(-(l + f) // ps) for l, f in zip(lens, fresh)) + 1
    held = [-(-l // ps) for l in lens]
    need = sum(-(-(l + f) // ps) - h for l, f, h in zip(lens, fresh, held))
    ids = r.permutation(sum(held) + need + spare + 2)
    tables = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for b, h in enumerate(held):
        tables[b, :h] = ids[at:at + h]
        at += h
    free = [int(v) for v in ids[at:]]
    return dict(lens=lens, fresh=fresh, free=free, pool=[2, len(free)], tables=tables,
                n=sum(fresh) + pad)


def run_tables(plan, c, base=0, in_place=False):
    lens, pool = ints(c["lens"]), ints(c["pool"])
    t = torch.from_numpy(c["tables"]).cuda()
    B = len(c["lens"])
    lens_out = lens if in_place else torch.full((B,), -9, dtype=torch.int32, device="cuda")
    pool_out = pool if in_place else torch.full((2,), -9, dtype=torch.int32, device="cuda")
    cu, pos, slots = ints([-9] * (B + 1)), ints([-9] * c["n"]), ints([-9] * c["n"])
    plan.build_tables(lens, ints(c["fresh"]), ints(c["free"]), pool, t, lens_out, pool_out, cu, pos,
                      slots, base=base)
    return [x.cpu().tolist() for x in (t, lens_out, pool_out, cu, pos, slots)]


def want_tables(c, ps, base=0):
    ok, t, lens, pool, cu, pos, slots = ref.build_tables(
        c["lens"], c["fresh"], c["free"], c["pool"], c["tables"], base, ps, c["n"])
    return ok, [t.tolist(), lens, pool, cu, pos, slots]


@pytest.mark.parametrize("B,ps,fresh", [(1, 16, 1), (3, 64, 5), (16, 16, 1), (33, 32, 90),
                                        (513, 16, 2), (1024, 192, 1), (1000, 64, 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_tables(cfa, B, ps, fresh, in_place):
    c = tables_case(B, ps, B, most_fresh=fresh)
    with cfa.Paged(B, 65536, 8, 2, 64, ps) as plan:
        for _ in range(2):  # the second call finds the arrival counter as the first left it
            ok, want = want_tables(c, ps, 1000)
            assert ok and run_tables(plan, c, 1000, in_place) == want
        assert plan.status() == cfa.CFA_OK


def test_tables_one_long_prompt(cfa):
    c = dict(lens=[0, 7], fresh=[65000, 0], free=list(range(5000, 0, -1)), pool=[0, 5000],
             tables=np.full((2, 4100), -1, dtype=np.int32), n=65536)
    c["tables"][1, 0] = 5001
    with cfa.Paged(2, 65536, 8, 2, 64, 16) as plan:
        ok, want = want_tables(c, 16)
        assert ok and run_tables(plan, c) == want


@pytest.mark.parametrize("how,code", [("pages", 6), ("tokens", 1), ("width", 1), ("negative", 1),
                                      ("pool", 6), ("taken", 1)])
def test_tables_refused_whole(cfa, how, code):
    c = tables_case(9, 16, 4, most_fresh=40)
    good = dict(c)
    if how == "pages":
        c["free"] = c["free"][:3]
        c["pool"] = [2, 3]
    if how == "pool":  # the pool says more than the list holds
        c["free"] = c["free"][:3]
        c["pool"] = [2, 1000]
    if how == "tokens":
        c["n"] = sum(c["fresh"]) - 1
    if how == "width":
        c["tables"] = c["tables"][:, :2].copy()
    if how == "negative":
        c["lens"] = [-1] + c["lens"][1:]
    if how == "taken":
        c["pool"] = [-1, len(c["free"])]
    with cfa.Paged(9, 4096, 8, 2, 64, 16) as plan:
        got = run_tables(plan, c)
        assert got == [c["tables"].tolist(), c["lens"], c["pool"], [0] * 10, [0] * c["n"], [-1] * c["n"]]
        assert plan.status() == code
        assert run_tables(plan, good) == want_tables(good, 16)[1]
        assert plan.status() == cfa.CFA_OK


def test_tables_checks_arguments(cfa):
    c = tables_case(4, 16, 1)
    with cfa.Paged(3, 64, 8, 2, 64, 16) as plan:
        with pytest.raises(cfa.CfaError):
            run_tables(plan, c)          # more requests than the plan's
    with cfa.Paged(4, 64, 8, 2, 64, 16) as plan:
        lens, x = ints([1] * 4), ints([0] * 64)
        args = dict(lens=lens, fresh=ints([1] * 4), free_pages=ints([1, 2, 3]), pool=ints([0, 3]),
                    tables=ints([[0] * 4] * 4), lens_out=ints([0] * 4), pool_out=ints([0, 0]),
                    cu=ints([0] * 5), positions=ints([0] * 8), slots=ints([0] * 8))
        for name, t, err in (("fresh", lens.float(), TypeError), ("cu", ints([0] * 4), ValueError),
                             ("slots", ints([0] * 16)[::2], ValueError),
                             ("fresh", lens.cpu(), ValueError),
                             ("lens_out", args["fresh"], cfa.CfaError),
                             ("pool_out", x[:2], None), ("positions", args["slots"], cfa.CfaError)):
            if err is not None:
                with pytest.raises(err):
                    plan.build_tables(**{**args, name: t})
        with pytest.raises(cfa.CfaError):
            plan.build_tables(**{**args, "base": -1})
        with pytest.raises(cfa.CfaError):
            plan.build_tables(**{**args, "base": (1 << 31) - 8})
        assert plan.status() == cfa.CFA_OK


@pytest.mark.parametrize("bad", [-1, -(1 << 31), (1 << 31) - 1, 1 << 27])
def test_tables_bad_page_ids(cfa, bad):
    """A held page or a free one that no slot can name: slot -1, flagged, the rest as ever."""
    with cfa.Paged(2, 8, 2, 1, 64, 16) as plan:
        tables = ints([[bad, -7, -7], [3, -7, -7]])
        cu, pos, slots, lens, pool = ints([0] * 3), ints([7] * 8), ints([7] * 8), ints([14, 16]), ints([0, 2])
        plan.build_tables(lens, ints([4, 2]), ints([bad, 5]), pool, tables, lens, pool, cu, pos, slots)
        assert plan.status() == cfa.CFA_ERR_INVALID_ARG
        # the first request's tokens 14 and 15 lie in its held page, 16 and 17 in the first free one
        assert slots.tolist() == [-1, -1, -1, -1, 5 * 16, 5 * 16 + 1, -1, -1]
        assert pos.tolist() == [14, 15, 16, 17, 16, 17, 0, 0] and cu.tolist() == [0, 4, 6]
        assert tables.tolist() == [[bad, bad, -7], [3, 5, -7]]
        assert lens.tolist() == [18, 18] and pool.tolist() == [2, 2]
        assert plan.status() == cfa.CFA_OK


def test_describe(cfa):
    with cfa.Paged(2, 8, 4, 2, 64, 16) as plan:
        d = plan.describe()
        rows = 2 * 2 * 16 + 512 * d["num_sms"]
        assert d["workspace_bytes"] == rows * 4 * 66 and d["smem_bytes"] > 0 and d["page_size"] == 16


# --------------------------------------------------------------------- append


ROPES = [
    dict(),
    dict(interleaved=True),
    dict(rotary_dim=32),
    dict(rotary_dim=32, interleaved=True, scaling="by_parts", factor=8.0, original_ctx=1024,
         magnitude=1.2),
    dict(rotary_dim=16, scaling="linear", factor=3.0),
    dict(rotary_dim=0),
    dict(theta=500000.0, scaling="by_parts", factor=32.0, low_turns=1.0, high_turns=4.0,
         original_ctx=8192),
]


@pytest.mark.parametrize("rope", ROPES)
@pytest.mark.parametrize("T,nh,nkv,d,ps", [(1, 4, 4, 128, 16), (5, 6, 2, 64, 64), (37, 7, 1, 128, 32)])
def test_append(cfa, rope, T, nh, nkv, d, ps):
    n_pages = -(-T // ps) + 1
    qkv = normal(T, T, (nh + 2 * nkv) * d)
    q = qkv[:, :nh * d].unflatten(1, (nh, d))
    k = qkv[:, nh * d:(nh + nkv) * d].unflatten(1, (nkv, d))
    v = qkv[:, (nh + nkv) * d:].unflatten(1, (nkv, d))
    r = np.random.default_rng(T)
    pos = [int(x) for x in r.integers(0, 1 << 22, T)]
    pos[-1] = (1 << 22) - 1
    slots = [int(x) for x in r.permutation(n_pages * ps)[:T]]
    if T > 2:
        slots[1] = -1
    kp, vp = normal(2, n_pages, nkv, ps, d), normal(3, n_pages, nkv, ps, d)
    k0, v0 = f64(kp), f64(vp)
    q_out = torch.full((T, nh, d), 7.0, dtype=torch.bfloat16, device="cuda")
    with cfa.Paged(1, T, nh, nkv, d, ps) as plan:
        plan.set_rope(**rope)
        plan.append(q, k, v, ints(pos), ints(slots), kp, vp, q_out)
        assert plan.status() == cfa.CFA_OK
    rd = rope.get("rotary_dim", d)
    f = ref.frequencies(rope.get("theta", 10000.0), rd,
                        **{x: rope[x] for x in ("scaling", "factor", "low_turns", "high_turns", "original_ctx") if x in rope})
    m, inter = rope.get("magnitude", 1.0), rope.get("interleaved", False)
    want_q, want_k = (ref.rotate(f64(x), pos, f, inter, m) for x in (q, k))
    live = [t for t in range(T) if slots[t] >= 0]

    def near(got, want, x):
        size = np.abs(x).max(-1, keepdims=True) * 2 * m
        assert np.all(np.abs(got - want) <= H8 * np.abs(want) + 1e-6 * size)

    near(f64(q_out)[live], want_q[live], f64(q)[live])
    assert torch.all(q_out[[t for t in range(T) if slots[t] < 0]] == 7.0)
    got_k, got_v = f64(kp), f64(vp)
    for t in live:
        p, o = divmod(slots[t], ps)
        near(got_k[p, :, o], want_k[t], f64(k)[t])
        assert np.array_equal(got_v[p, :, o], f64(v)[t])
        got_k[p, :, o], got_v[p, :, o] = k0[p, :, o], v0[p, :, o]
    assert np.array_equal(got_k, k0) and np.array_equal(got_v, v0)


def test_append_in_place_and_bad_slots(cfa):
    T, nh, d = 6, 4, 64
    q, k, v = normal(1, T, nh, d), normal(2, T, nh, d), normal(3, T, nh, d)
    kp, vp = normal(4, 2, nh, 16, d), normal(5, 2, nh, 16, d)
    pos = ints(range(T))
    with cfa.Paged(1, T, nh, nh, d, 16) as plan:
        plan.set_rope()
        other = torch.empty_like(q)
        plan.append(q, k, v, pos, ints([0, 1, 2, 3, 4, 31]), kp, vp, other)
        k1, v1, mine = kp.clone(), vp.clone(), q.clone()
        plan.append(mine, k, v, pos, ints([0, 1, 2, 3, 4, 31]), kp, vp, mine)
        assert torch.equal(mine, other) and torch.equal(kp, k1) and torch.equal(vp, v1)
        assert plan.status() == cfa.CFA_OK
        plan.append(q, k, v, pos, ints([0, 1, 2, 3, 32, 2**31 - 1]), kp, vp, torch.empty_like(q))
        assert torch.equal(kp, k1) and torch.equal(vp, v1)
        assert plan.status() == cfa.CFA_ERR_INVALID_ARG
        # no tokens at all
        plan.append(q[:0], k[:0], v[:0], pos[:0], pos[:0], kp, vp, q[:0].clone())
        assert plan.status() == cfa.CFA_OK


def test_append_most_tokens_far_apart(cfa):
    """The most tokens a plan takes, in rows that lie beyond 2^32 elements."""
    T, d, ps = 1 << 17, 64, 64
    rows = torch.empty(T, 1 << 15, dtype=torch.bfloat16, device="cuda")[:, :3 * d]
    rows.copy_(normal(1, T, 3 * d))
    dense = rows.contiguous()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.flip(pos, (0,)).contiguous()
    got = []
    with cfa.Paged(1, T, 1, 1, d, ps) as plan:
        plan.set_rope()
        for x in (rows, dense):
            kp, vp = (torch.zeros(T // ps, 1, ps, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            q = torch.zeros(T, 1, d, dtype=torch.bfloat16, device="cuda")
            plan.append(x[:, :d].unsqueeze(1), x[:, d:2 * d].unsqueeze(1), x[:, 2 * d:].unsqueeze(1), pos, slots,
                        kp, vp, q)
            got.append((q, kp, vp))
        assert plan.status() == cfa.CFA_OK
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert torch.equal(got[0][2].view(T, d), torch.flip(dense[:, 2 * d:], (0,)))
    some = [0, 1, T // 2, T - 1]
    x = f64(dense[some])
    want = ref.rotate(x[:, None, d:2 * d], some, ref.frequencies(10000.0, d), False)[:, 0]
    k = f64(got[0][1].view(T, d)[[T - 1 - t for t in some]])
    assert np.all(np.abs(k - want) <= H8 * np.abs(want) + 1e-6 * 2 * np.abs(x).max())


def test_append_checks_arguments(cfa):
    T, nh, d = 4, 4, 64
    q, k, v = normal(1, T, nh, d), normal(2, T, 2, d), normal(3, T, 2, d)
    kp, vp = normal(4, 2, 2, 16, d), normal(5, 2, 2, 16, d)
    a = dict(q=q, k=k, v=v, positions=ints([0] * T), slots=ints(range(T)), k_pages=kp, v_pages=vp,
             q_out=torch.empty_like(q))
    wide = normal(6, T, nh * d + 4)
    for name, t, err in (("q", q.float(), TypeError), ("q", q.transpose(0, 1), ValueError),
                         ("q", wide[:, 4:].unflatten(1, (nh, d)), cfa.CfaError),
                         ("k", q, ValueError), ("v_pages", kp, cfa.CfaError),
                         ("q_out", q.reshape(-1)[: T * nh * d].view(T, nh, d), None),
                         ("k_pages", kp[:, :, ::2], ValueError), ("slots", ints([0] * 3), ValueError)):
        with cfa.Paged(1, T, nh, 2, d, 16) as plan:
            if err is None:
                plan.append(**{**a, name: t})
            else:
                with pytest.raises(err):
                    plan.append(**{**a, name: t})
    fused = normal(7, T, (nh + 4) * d)
    with cfa.Paged(1, T, nh, 2, d, 16) as plan:
        with pytest.raises(cfa.CfaError):  # an output over a strided input
            plan.append(**{**a, "q": fused[:, :nh * d].unflatten(1, (nh, d)),
                           "q_out": fused.view(-1)[: T * nh * d].view(T, nh, d)})
        with pytest.raises(cfa.CfaError):
            plan.set_rope(rotary_dim=24)
        with pytest.raises(cfa.CfaError):
            plan.set_rope(rotary_dim=80)
        with pytest.raises(cfa.CfaError):
            plan.set_rope(theta=0.5)
        with pytest.raises(cfa.CfaError):
            plan.set_rope(scaling="by_parts", low_turns=2.0, high_turns=2.0)
        with pytest.raises(ValueError):
            plan.set_rope(scaling="other")
        with pytest.raises(cfa.CfaError):
            plan.set_rope(factor=float("nan"), scaling="linear")
    with cfa.Paged(1, T - 1, nh, 2, d, 16) as plan:
        with pytest.raises(cfa.CfaError):
            plan.append(**a)


# ------------------------------------------------------------------ attention


def attn_case(seed, nh, nkv, d, ps, prefix, lens, news, poison=True, spiky=False):
    r = np.random.default_rng(seed)
    held = [-(-l // ps) for l in lens]
    n_prefix = -(-prefix // ps)
    width = max(max(held), 1) + 1
    n_pages = n_prefix + sum(held) + 2
    ids = [int(v) for v in r.permutation(n_pages)]
    kp, vp = normal(seed + 1, n_pages, nkv, ps, d), normal(seed + 2, n_pages, nkv, ps, d)
    if spiky:
        kp[torch.rand(n_pages, nkv, ps, device="cuda") < 0.05] *= 4
    tables = np.full((len(lens), width), n_pages + 7, dtype=np.int32)  # never looked up
    used = torch.zeros(n_pages, ps, dtype=torch.bool)
    for j in range(n_prefix):
        used[ids[j], :min(ps, prefix - j * ps)] = True
    at = n_prefix
    for b, h in enumerate(held):
        tables[b, :h] = ids[at:at + h]
        for j in range(h):
            used[ids[at + j], :min(ps, lens[b] - j * ps)] = True
        at += h
    if poison:
        hole = ~used.cuda()
        kp.transpose(1, 2)[hole] = float("nan")
        vp.transpose(1, 2)[hole] = float("nan")
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    return dict(q=normal(seed + 3, cu[-1], nh, d), kp=kp, vp=vp, tables=tables, lens=list(lens),
                cu=cu, prefix_table=ids[:n_prefix], prefix=prefix, ps=ps)


def attend(plan, c, q=None, scale=None, out=None, lse=None, stream=None):
    q = c["q"] if q is None else q
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    lse = torch.full(q.shape[:2], 7.0, device="cuda") if lse is None else lse
    plan.attend(q, ints(c["cu"]), ints(c["lens"]), torch.from_numpy(c["tables"]).cuda(), c["kp"],
                c["vp"], out, prefix_table=ints(c["prefix_table"]) if c["prefix"] else None,
                prefix_len=c["prefix"], scale=scale, lse=lse, stream=stream)
    return out, lse


def check_attn(c, out, lse, scale=None):
    want, want_lse, size = ref.attention(f64(c["q"]), c["cu"], c["lens"], c["tables"], f64(c["kp"]),
                                         f64(c["vp"]), c["prefix_table"], c["prefix"], scale)
    got, got_lse = f64(out), f64(lse)
    rows = slice(c["cu"][0], c["cu"][-1])
    tol = (1 + 2.0 ** -4) * H8 * (np.abs(want) + size) + 1e-6
    off = np.abs(got - want)[rows] - tol[rows]
    assert np.all(off <= 0), (float(off.max()), np.unravel_index(off.argmax(), off.shape))
    empty = np.isneginf(want_lse[rows])
    assert np.array_equal(np.isneginf(got_lse[rows]), empty)
    assert np.all(np.abs(got_lse[rows][~empty] - want_lse[rows][~empty]) <= 1e-4)


ATTN = [
    # nh, nkv, d, ps, prefix, lens, new tokens
    (2, 2, 128, 64, 0, [1], [1]),                             # one key
    (4, 4, 128, 64, 64, [64], [1]),
    (4, 2, 128, 16, 1, [1, 17, 33], [1, 1, 1]),
    (2, 1, 64, 32, 127, [1, 200, 31], [1, 1, 1]),
    (8, 2, 128, 64, 129, [128, 129, 127, 1], [1, 1, 1, 1]),
    (7, 1, 64, 128, 300, [5, 260], [1, 1]),                   # a group of 7
    (32, 2, 64, 192, 200, [400, 20], [1, 1]),                 # a group of 16, pages of 3 x 64
    (40, 2, 128, 64, 70, [90, 3], [1, 1]),                    # a group above 16
    (8, 2, 128, 32, 513, [40, 8, 9, 300], [8, 8, 1, 5]),      # drafted tokens
    (4, 1, 128, 64, 100, [200, 70], [130, 70]),               # prompt chunks
    (8, 1, 64, 16, 257, [300, 64, 1], [300, 40, 1]),
    (2, 2, 128, 64, 0, [0, 3, 0], [1, 1, 2]),                 # rows without keys
    (2, 2, 64, 64, 33, [0, 3, 2], [1, 0, 5]),                 # no rows, no keys, more rows than keys
    (1, 1, 128, 16, 1500, [700] * 5, [1] * 5),                # split over many blocks
    (16, 16, 64, 64, 1000, [250, 1, 600], [1, 1, 1]),
    (4, 4, 128, 64, 640, [33] * 40, [1] * 40),                # 40 rows a key head
    (8, 2, 128, 16, 300, [20] * 70, [1] * 70),                # 280 rows a key head: two row tiles
    (4, 1, 64, 64, 130, [64 + i for i in range(150)], [1] * 150),
    (2, 1, 128, 4096, 100, [4000], [1]),                      # a whole cache as one page
    (16, 16, 64, 64, 4000, [9000, 8500, 300], [1, 1, 1]),     # several long pieces to a block
    (8, 8, 128, 64, 2500, [12000, 700, 11000, 40], [1, 1, 1, 1]),
    (16, 4, 128, 64, 6000, [9000, 8000, 2000, 5000], [9, 1, 1, 6]),  # few rows and tiles in turn
    (16, 4, 64, 32, 3000, [9000, 200, 7000, 5000], [1, 7, 40, 1]),
]


@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention(cfa, case):
    nh, nkv, d, ps, prefix, lens, news = ATTN[case]
    c = attn_case(100 + case, nh, nkv, d, ps, prefix, lens, news)
    with cfa.Paged(len(lens), sum(news), nh, nkv, d, ps) as plan:
        out, lse = attend(plan, c)
        again, lse2 = attend(plan, c)
        assert plan.status() == cfa.CFA_OK
    check_attn(c, out, lse)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("seed", range(12))
def test_attention_random_shapes(cfa, seed):
    r = np.random.default_rng(seed)
    nkv, G = int(r.integers(1, 4)), int(r.choice([1, 2, 3, 4, 8, 12, 16, 20]))
    d, ps = int(r.choice([64, 128])), int(r.choice([16, 32, 64, 128, 320]))
    B = int(r.integers(1, 7))
    lens = [int(x) for x in r.integers(0, 400, B)]
    news = [int(x) for x in r.integers(0, int(r.choice([2, 6, 40])), B)]
    news[0] = max(1, news[0])
    c = attn_case(seed, nkv * G, nkv, d, ps, int(r.integers(0, 900)), lens, news, spiky=seed % 2 == 0)
    scale = None if seed % 3 else 0.3
    with cfa.Paged(B + 3, sum(news) + 9, nkv * G, nkv, d, ps) as plan:
        out, lse = attend(plan, c, scale=scale)
        assert plan.status() == cfa.CFA_OK
    check_attn(c, out, lse, scale)


TILES = [
    # nh, nkv, d, ps, prefix, lens, new tokens
    (8, 1, 128, 64, 200, [300, 150], [12, 9]),                # 96 and 72 rows: one tile over own keys
    (8, 1, 64, 32, 0, [500, 77, 40, 9], [16, 3, 7, 17]),      # 128, 24, 56, and 136 rows
    (3, 1, 128, 16, 90, [64, 65, 20], [21, 20, 22]),          # 63, 60 and 66 rows
    (16, 2, 128, 64, 300, [700, 513], [100, 65]),             # 800 and 520 rows: several tiles each
    (16, 1, 64, 16, 0, [70, 300], [70, 17]),                  # the same without a prefix
    (4, 4, 64, 64, 700, [i % 5 for i in range(600)], [1] * 600),         # three tiles over the prefix
    (2, 1, 64, 16, 33, [i % 40 for i in range(1024)], [i % 3 for i in range(1024)]),
    (2, 1, 128, 32, 0, [1 + i % 70 for i in range(1024)], [1] * 1024),
    (128, 1, 128, 64, 150, [70, 1], [1, 1]),                  # a group of 128: the most that shares
    (129, 1, 64, 64, 150, [70, 1], [1, 1]),                   # and one more
    (1024, 2, 64, 64, 20, [9], [1]),
]


@pytest.mark.parametrize("case", range(len(TILES)))
def test_attention_tiles(cfa, case):
    nh, nkv, d, ps, prefix, lens, news = TILES[case]
    c = attn_case(300 + case, nh, nkv, d, ps, prefix, lens, news)
    with cfa.Paged(len(lens), sum(news), nh, nkv, d, ps) as plan:
        out, lse = attend(plan, c)
        assert plan.status() == cfa.CFA_OK
    check_attn(c, out, lse)


@pytest.mark.parametrize("n,own,prefix,nh,nkv,d", [
    (5000, 6001, 300, 8, 2, 128),          # a long prompt: many tiles, each cut by a run's end at most once
    (1, 1 << 20, 0, 4, 1, 64),             # one row over a million keys: every run has a piece of it
    (2, 70, 1 << 19, 2, 1, 128),           # and over a long prefix
    (1 << 17, 40, 9, 1, 1, 64),            # the most tokens, most of them without own keys
])
def test_attention_long(cfa, n, own, prefix, nh, nkv, d):
    """The largest calls, a few rows of each against 64 bits."""
    ps, np_ = 64, -(-prefix // 64)
    pages = np_ + -(-own // ps)
    kp, vp = normal(1, pages, nkv, ps, d), normal(2, pages, nkv, ps, d)
    c = dict(q=normal(3, n, nh, d), kp=kp, vp=vp, tables=np.arange(np_, pages, dtype=np.int32)[None].copy(),
             lens=[own], cu=[0, n], prefix_table=list(range(np_)), prefix=prefix)
    with cfa.Paged(1, n, nh, nkv, d, ps) as plan:
        out, lse = attend(plan, c)
        assert plan.status() == cfa.CFA_OK
    for i in {0, 1 % n, n // 3, max(0, n - own), n - 1}:
        see = min(own, max(0, own - n + i + 1))
        for h in {0, nh - 1}:
            g = h * nkv // nh
            k, v = (torch.cat((x[:np_, g].reshape(-1, d)[:prefix], x[np_:, g].reshape(-1, d)[:see])).double()
                    for x in (kp, vp))
            s = k @ c["q"][i, h].double() / math.sqrt(d)
            w = torch.softmax(s, 0)
            want, size = w @ v, w @ v.abs()
            tol = (1 + 2.0 ** -4) * H8 * (want.abs() + size) + 1e-6
            assert torch.all((out[i, h].double() - want).abs() <= tol)
            assert abs(float(lse[i, h]) - float(torch.logsumexp(s, 0))) <= 1e-4


def test_attention_far_pages_and_rows(cfa):
    """Pages beyond 2^32 elements of their cache, query rows as far behind the first."""
    nh, nkv, d, ps, pages = 8, 8, 128, 64, 70000
    c = attn_case(12, nh, nkv, d, ps, 100, [130, 70, 3], [2, 1, 1])
    n, T = c["kp"].shape[0], c["q"].shape[0]
    kp, vp = (torch.empty(pages, nkv, ps, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kp[pages - n:], vp[pages - n:] = c["kp"], c["vp"]
    far = dict(c, kp=kp, vp=vp, tables=(c["tables"] + (pages - n)).astype(np.int32),
               prefix_table=[i + pages - n for i in c["prefix_table"]])
    q = torch.empty(T, 1 << 31, dtype=torch.bfloat16, device="cuda")[:, :nh * d].unflatten(1, (nh, d))
    q.copy_(c["q"])
    with cfa.Paged(3, T, nh, nkv, d, ps) as plan:
        out, lse = attend(plan, far, q=q)
        assert plan.status() == cfa.CFA_OK
        check_attn(c, out, lse)
        k, v = normal(1, T, nkv, d), normal(2, T, nkv, d)
        slots = [pages * ps - 1, (pages - n) * ps, pages * ps - 2, -1]
        plan.append(q, k, v, ints([0] * T), ints(slots), kp, vp, torch.empty_like(out))
        assert plan.status() == cfa.CFA_OK
        for t, s in enumerate(slots[:3]):
            assert torch.equal(kp[s // ps, :, s % ps], k[t]) and torch.equal(vp[s // ps, :, s % ps], v[t])


def test_two_graphs_of_one_plan(cfa):
    """Graphs of different batches take turns in the plan's workspace."""
    cases = [attn_case(13, 8, 2, 64, 32, 400, [300, 10, 99], [1, 3, 40]),
             attn_case(14, 8, 2, 64, 32, 0, [900] * 4, [1] * 4),
             attn_case(15, 8, 2, 64, 32, 1300, [1], [1])]
    with cfa.Paged(4, 44, 8, 2, 64, 32) as plan:
        want = [attend(plan, c) for c in cases]
        graphs, got = [], []
        for c in cases:
            a = (c["q"], ints(c["cu"]), ints(c["lens"]), torch.from_numpy(c["tables"]).cuda(), c["kp"], c["vp"])
            out, lse = torch.zeros_like(c["q"]), torch.zeros(c["q"].shape[:2], device="cuda")
            pt = ints(c["prefix_table"]) if c["prefix"] else None
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                plan.attend(*a, out, prefix_table=pt, prefix_len=c["prefix"], lse=lse)
            graphs.append((g, a, pt))
            got.append((out, lse))
        for turn in (0, 1, 2, 2, 1, 0, 2, 0):
            for x in got[turn]:
                x.zero_()
            graphs[turn][0].replay()
            attend(plan, cases[(turn + 1) % 3])
            assert all(torch.equal(x, y) for x, y in zip(got[turn], want[turn]))
        assert plan.status() == cfa.CFA_OK


def test_attention_extreme_scores(cfa):
    """Scores of some thousands, equal and opposite, and a key far above the others."""
    c = attn_case(5, 4, 2, 64, 64, 200, [150, 9], [3, 1], poison=False)
    c["q"] *= 64
    c["kp"] *= 16
    c["kp"][:, :, 3] = -c["kp"][:, :, 2]
    with cfa.Paged(2, 4, 4, 2, 64, 64) as plan:
        out, lse = attend(plan, c)
    want, want_lse, size = ref.attention(f64(c["q"]), c["cu"], c["lens"], c["tables"], f64(c["kp"]),
                                         f64(c["vp"]), c["prefix_table"], c["prefix"])
    # a score is off by up to d 2^-24 sum |q k| scale, here 64 2^-24 (64 * 64 * 16 * 4) / 8 < 0.13,
    # and every weight by that factor
    tol = H8 * (np.abs(want) + size) * 1.1 + 2 * 0.13 * size
    assert np.all(np.isfinite(f64(out))) and np.all(np.abs(f64(out) - want) <= tol)
    assert np.all(np.abs(f64(lse) - want_lse) <= 0.13 + 2.0 ** -22 * np.abs(want_lse))


def test_attention_leaves_other_rows(cfa):
    c = attn_case(6, 8, 2, 128, 64, 140, [70, 9, 30], [2, 1, 30])
    q = torch.cat((normal(1, 2, 8, 128), c["q"], normal(2, 3, 8, 128)))
    c = dict(c, q=q, cu=[x + 2 for x in c["cu"]])
    with cfa.Paged(3, 64, 8, 2, 128, 64) as plan:
        out, lse = attend(plan, c)
    check_attn(c, out, lse)
    for t in (out, lse):
        assert torch.all(t[:2] == 7.0) and torch.all(t[-3:] == 7.0)


def test_attention_reads_strided_q(cfa):
    c = attn_case(7, 8, 2, 64, 32, 140, [70, 9], [1, 20])
    T = c["q"].shape[0]
    fused = normal(3, T, 8 * 64 + 256)
    fused[:, :512] = c["q"].reshape(T, 512)
    with cfa.Paged(2, T, 8, 2, 64, 32) as plan:
        a, la = attend(plan, c)
        b, lb = attend(plan, c, q=fused[:, :512].unflatten(1, (8, 64)))
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("cu", [[0, 3, 2], [-1, 1, 2], [0, 1, 9], [0, 2, 1 << 30]])
def test_attention_bad_offsets_write_nothing(cfa, cu):
    c = attn_case(8, 4, 2, 64, 64, 70, [40, 30], [2, 1])
    with cfa.Paged(2, 8, 4, 2, 64, 64) as plan:
        good, _ = attend(plan, c)
        out, lse = attend(plan, dict(c, cu=cu))
        assert torch.all(out == 7.0) and torch.all(lse == 7.0)
        assert plan.status() == cfa.CFA_ERR_INVALID_ARG
        assert torch.equal(attend(plan, c)[0], good)
        assert plan.status() == cfa.CFA_OK


@pytest.mark.parametrize("G,new", [(1, 1), (4, 9)])
@pytest.mark.parametrize("bad", [-1, 1 << 20, -(1 << 31), (1 << 31) - 1])
def test_attention_bad_pages_and_lengths(cfa, bad, G, new):
    """A page id outside the cache reads as zeros, a length outside the table as 0."""
    c = attn_case(9, 2 * G, 2, 128, 32, 100, [70, 90], [new, new])
    c["tables"] = c["tables"].copy()
    c["tables"][0, 1] = bad
    c["prefix_table"] = c["prefix_table"][:2] + [bad] + c["prefix_table"][3:]
    with cfa.Paged(2, 2 * new, 2 * G, 2, 128, 32) as plan:
        out, lse = attend(plan, c)
        assert plan.status() == cfa.CFA_ERR_INVALID_ARG
        check_attn(c, out, lse)
        c = attn_case(9, 2 * G, 2, 128, 32, 100, [70, 90], [new, new])
        out, lse = attend(plan, dict(c, lens=[bad, 90]))
        assert plan.status() == cfa.CFA_ERR_INVALID_ARG
        check_attn(dict(c, lens=[0, 90]), out, lse)


def test_attention_checks_arguments(cfa):
    c = attn_case(10, 4, 2, 64, 64, 70, [40, 30], [2, 1])
    a = dict(q=c["q"], cu=ints(c["cu"]), lens=ints(c["lens"]), tables=torch.from_numpy(c["tables"]).cuda(),
             k_pages=c["kp"], v_pages=c["vp"], out=torch.empty_like(c["q"]),
             prefix_table=ints(c["prefix_table"]), prefix_len=70)
    with cfa.Paged(2, 4, 4, 2, 64, 64) as plan:
        for name, t, err in (("q", c["q"].half(), TypeError), ("cu", ints([0, 1]), ValueError),
                             ("lens", a["lens"].long(), TypeError), ("out", c["q"], cfa.CfaError),
                             ("prefix_table", None, ValueError), ("prefix_len", 129, ValueError),
                             ("prefix_len", -1, ValueError), ("scale", -1.0, ValueError),
                             ("scale", float("nan"), ValueError), ("scale", float("inf"), cfa.CfaError),
                             ("lse", torch.empty(3, 3, device="cuda"), ValueError),
                             ("tables", a["tables"][0], ValueError),
                             ("k_pages", c["kp"][:, :1], ValueError)):
            with pytest.raises(err):
                plan.attend(**{**a, name: t})
        plan.attend(**a)
        plan.attend(**{**a, "q": c["q"][:0], "out": c["q"][:0].clone()})
        assert plan.status() == cfa.CFA_OK
    with cfa.Paged(1, 4, 4, 2, 64, 64) as plan:
        with pytest.raises(cfa.CfaError):
            plan.attend(**a)


def test_attention_on_another_stream_and_two_plans(cfa):
    c = attn_case(11, 8, 2, 128, 64, 700, [300, 10, 99], [1, 3, 40])
    with cfa.Paged(3, 44, 8, 2, 128, 64) as one, cfa.Paged(3, 44, 8, 2, 128, 64) as two:
        want, _ = attend(one, c)
        torch.cuda.synchronize()
        s, t = torch.cuda.Stream(), torch.cuda.Stream()
        outs = []
        for _ in range(4):
            with torch.cuda.stream(s):
                outs.append(attend(one, c)[0])
            with torch.cuda.stream(t):
                outs.append(attend(two, c)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)


# ------------------------------------------------------------------- together


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("nh,nkv,d,ps", [(8, 2, 128, 16), (4, 4, 64, 64)])
def test_decode_loop(cfa, nh, nkv, d, ps, graph):
    """Steps of a ragged batch: tables, then two layers of append and attention, the
    lengths and the pool advancing in place; as one recorded graph or call by call."""
    B, P, T, layers, steps, pages = 5, 75, 24, 2, 4, 64
    r = np.random.default_rng(3)
    n_prefix = -(-P // ps)
    ids = [int(x) for x in r.permutation(pages)]
    prefix_table, free = ids[:n_prefix], ids[n_prefix:]
    width = 8
    news = [[int(x) for x in r.integers(0, 5, B)] for _ in range(steps)]
    caches = [(normal(20 + i, pages, nkv, ps, d), normal(30 + i, pages, nkv, ps, d)) for i in range(layers)]
    model = [(f64(k), f64(v)) for k, v in caches]
    lens, pool, tables = ints([0] * B), ints([0, len(free)]), torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    fresh, freet, pt = ints([0] * B), ints(free), ints(prefix_table)
    cu, pos, slots = ints([0] * (B + 1)), ints([0] * T), ints([0] * T)
    qkv = [torch.zeros(T, (nh + 2 * nkv) * d, dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
    outs = [torch.zeros(T, nh, d, dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
    turned = torch.zeros(T, nh, d, dtype=torch.bfloat16, device="cuda")
    rope = dict(rotary_dim=d // 2, interleaved=True)
    with cfa.Paged(B, T, nh, nkv, d, ps) as plan:
        plan.set_rope(**rope)

        def step():
            plan.build_tables(lens, fresh, freet, pool, tables, lens, pool, cu, pos, slots, base=P)
            for x, (kp, vp), o in zip(qkv, caches, outs):
                q, k, v = x.split((nh * d, nkv * d, nkv * d), 1)
                plan.layer(q.unflatten(1, (nh, d)), k.unflatten(1, (nkv, d)), v.unflatten(1, (nkv, d)),
                           pos, slots, cu, lens, tables, kp, vp, turned, o, prefix_table=pt, prefix_len=P)

        g = None
        if graph:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                step()
        host_lens, host_pool = [0] * B, [0, len(free)]
        host_tables = np.full((B, width), -1, dtype=np.int32)
        for n, new in enumerate(news):
            fresh.copy_(ints(new))
            for i, x in enumerate(qkv):
                x.copy_(normal(100 * n + i, *x.shape))
            g.replay() if graph else step()
            assert plan.status() == cfa.CFA_OK
            ok, host_tables, host_lens, host_pool, host_cu, host_pos, host_slots = ref.build_tables(
                host_lens, new, free, host_pool, host_tables, P, ps, T)
            assert ok and cu.tolist() == host_cu and slots.tolist() == host_slots
            assert lens.tolist() == host_lens and pool.tolist() == host_pool
            total, f = host_cu[-1], ref.frequencies(10000.0, d // 2)
            for x, (mk, mv), (kp, vp), o in zip(qkv, model, caches, outs):
                q, k, v = (f64(y) for y in x.split((nh * d, nkv * d, nkv * d), 1))
                q = ref.rotate(q.reshape(T, nh, d), host_pos, f, True)
                k, v = ref.rotate(k.reshape(T, nkv, d), host_pos, f, True), v.reshape(T, nkv, d)
                for t in range(total):
                    p, off = divmod(host_slots[t], ps)
                    mk[p, :, off], mv[p, :, off] = k[t], v[t]
                assert np.all(np.abs(f64(kp) - mk) <= H8 * np.abs(mk) + 1e-5)
                want, _, size = ref.attention(q, host_cu, host_lens, host_tables, mk, mv, prefix_table, P)
                got = f64(o)[:total]
                # as above, and q and k rounded to bf16 after the rotation: a score is off by up to
                # 2 * 2^-8 sum |q k| / sqrt(d), about 2^-7 * 0.64 * 0.64 * sqrt(d), each weight by that
                lim = H8 * 1.1 * (np.abs(want) + size) + 2.0 ** -7 * 0.41 * math.sqrt(d) * 2 * size + 1e-6
                assert np.all(np.abs(got - want[:total]) <= lim[:total])


def test_reads_the_fused_blocks_cache(cfa):
    """A contiguous cache that the fused decode block filled, read as pages of max_ctx rows."""
    from out_proj_block_gb300 import workloads
    wl = workloads.WORKLOADS["tiny"]
    t = workloads.make_inputs(wl, seed=0, device="cuda:0", poison_tail=True)
    out = torch.empty(wl.B, wl.hidden, dtype=torch.bfloat16, device="cuda")
    with cfa.Plan(wl.B, wl.hidden, wl.n_heads, wl.head_dim, wl.max_ctx) as plan:
        plan.decode_step(t["x"], t["W_qkv"], t["W_o"], t["k_cache"], t["v_cache"], wl.ctx_len, out)
    c = dict(q=normal(1, wl.B, wl.n_heads, wl.head_dim), kp=t["k_cache"], vp=t["v_cache"],
             tables=np.arange(wl.B, dtype=np.int32)[:, None].copy(), lens=[wl.ctx_len + 1] * wl.B,
             cu=list(range(wl.B + 1)), prefix_table=[], prefix=0, ps=wl.max_ctx)
    with cfa.Paged(wl.B, wl.B, wl.n_heads, wl.n_heads, wl.head_dim, wl.max_ctx) as plan:
        got, lse = attend(plan, c)
    check_attn(c, got, lse)
