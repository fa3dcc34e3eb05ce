"""Paged latent-cache operators on the GPU against their fp64 definitions.

Tolerances, from the roundings alone (a bf16 rounding is at most 2^-8 of the value):
  append     one rounding of y: 2^-8 |y|; the norm (512 squares summed in fp32) and the
             angles add less than 2^-18 of the value's or the pair's magnitude.
  fold,      one rounding, 2^-8 |y|, and fp32 sums of n = 128 or 512 products: n 2^-24 sum |x w|.
  unfold
  attention  the weights are rounded to bf16 for their product with the values (2^-8 each, so at most
             2^-8 sum w|v| / sum w), the result once more (2^-8 |o|). A score of d = 576 or 192
             products in fp32 is off by at most d 2^-24 sum |q k| scale, a weight by that part of
             itself: with sum |q k| scale below 50 here, 2^-9 at worst and, as the errors of its
             products do not all agree in sign, far below 2^-12 in fact; the tests allow a sixteenth
             of 2^-8. lse: 1e-4 for scores of such sizes.
"""
import math

import numpy as np
import pytest
import torch

from oracle import cfa_oracle_latent as ref
from oracle import cfa_oracle_paged

pytestmark = pytest.mark.gpu

H8 = 2.0 ** -8
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


def weights(seed, H):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(C, H * 256, generator=g, device="cuda") / math.sqrt(C)).to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


def same_bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def close(got, want, size, what=""):
    tol = H8 * (size * 1.0625 + np.abs(want)) + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(got - want) / tol)} at {np.argwhere(bad)[:3].tolist()}"


# --------------------------------------------------------------------- append


ROPES = [dict(), dict(interleaved=True), dict(scaling="linear", factor=4.0),
         dict(interleaved=True, scaling="by_parts", factor=40.0, magnitude=1.25)]


def freqs(rope):
    r = {k: v for k, v in rope.items() if k not in ("interleaved", "magnitude")}
    return cfa_oracle_paged.frequencies(r.pop("theta", 10000.0), 64, **r)


@pytest.mark.parametrize("T,H,ps,rope", [(1, 1, 16, 0), (3, 128, 64, 1), (65, 31, 32, 2), (130, 33, 128, 3),
                                         (2, 64, 192, None), (7, 5, 16, 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_append(cfa, T, H, ps, rope, in_place):
    pages = normal(1, T // ps + 3, ps, ROW)
    wide = normal(2, T, 100 * 8 + ROW)
    a = wide[:, 800:]
    q = normal(3, T, H, QK) if in_place else normal(3, T, H * QK + 40)[:, 8:8 + H * QK].unflatten(1, (H, QK))
    g = (1.0 + 0.2 * normal(4, C).float()).to(torch.bfloat16)
    r = np.random.default_rng(5)
    pos = [int(v) for v in r.integers(0, 1 << 22, T)]
    slots = [int(v) for v in r.permutation(pages.shape[0] * ps)[:T]]
    if T > 2:
        slots[1] = -1  # skipped
    spec = ROPES[rope] if rope is not None else None
    before, q_in = pages.clone(), q.clone()
    q_out = q if in_place else torch.full((T, H, QK), 7.0, dtype=torch.bfloat16, device="cuda")
    kept = q_out.clone()
    with cfa.Latent(4, 256, H, ps) as plan:
        if spec is not None:
            plan.set_rope(**spec)
        assert plan.append(a, g, q, ints(pos), ints(slots), pages, q_out, eps=1e-5) is q_out
        assert plan.status() == cfa.CFA_OK
    args = (None,) if spec is None else (freqs(spec), spec.get("interleaved", False), spec.get("magnitude", 1.0))
    want_rows, want_q = ref.rows(f64(a), f64(g), 1e-5, pos, *args), ref.queries(f64(q_in), pos, *args)
    flat, was = f64(pages).reshape(-1, ROW), f64(before).reshape(-1, ROW)
    live = np.array([s >= 0 for s in slots])
    want = was.copy()
    for t in range(T):
        if live[t]:
            want[slots[t]] = want_rows[t]
    m = 1.0 if spec is None else spec.get("magnitude", 1.0)
    near = lambda got, want, size: np.all(np.abs(got - want) <= H8 * np.abs(want) + 2.0 ** -18 * size)  # noqa: E731
    assert near(flat, want, np.abs(want) + 4.0 * m * (np.arange(ROW) >= C))
    untouched = np.ones(len(flat), dtype=bool)
    untouched[[s for s in slots if s >= 0]] = False
    assert np.array_equal(flat[untouched], was[untouched])
    got = f64(q_out)
    assert near(got[live], want_q[live], 4.0 * m * (np.arange(QK) >= 128))
    assert np.array_equal(got[live][..., :128], want_q[live][..., :128])
    assert same_bits(q_out[torch.tensor(~live)], kept[torch.tensor(~live)])
    if spec is None:
        assert np.array_equal(flat[[s for s in slots if s >= 0], C:], f64(a)[live, C:])


def test_append_flags_a_far_slot(cfa):
    pages, q = normal(1, 2, 16, ROW), normal(2, 2, 3, QK)
    was, q_out = pages.clone(), torch.zeros_like(q)
    with cfa.Latent(1, 4, 3, 16) as plan:
        plan.append(normal(3, 2, ROW), normal(4, C), q, ints([0, 1]), ints([32, -5]), pages, q_out)
        assert plan.status() == cfa.CFA_ERR_INVALID_ARG
        assert plan.status() == cfa.CFA_OK
    assert same_bits(pages, was) and not q_out.any()


def test_append_of_zeros_and_not_finite(cfa):
    """A row of zeros is zeros (eps > 0); a value that is not finite stays in its token."""
    a = normal(1, 3, ROW)
    a[0] = 0
    a[1, 5] = float("inf")
    pages, q = torch.zeros(1, 16, ROW, dtype=torch.bfloat16, device="cuda"), normal(2, 3, 2, QK)
    with cfa.Latent(1, 4, 2, 16) as plan:
        plan.set_rope()
        plan.append(a, torch.ones(C, dtype=torch.bfloat16, device="cuda"), q, ints([1, 2, 3]), ints([0, 1, 2]),
                    pages, q)
    x = f64(pages)[0]
    assert not x[0].any() and not np.isfinite(x[1, 5]) and np.isfinite(x[2:]).all()


# ------------------------------------------------------------- fold and unfold


@pytest.mark.parametrize("T,H", [(1, 1), (1, 128), (2, 3), (4, 20), (15, 7), (16, 8), (17, 33), (63, 2), (65, 5),
                                 (129, 4), (300, 3),
                                 # many tokens by heads, and either side of where the form changes
                                 (33, 128), (48, 128), (49, 128), (20, 80), (21, 96), (128, 50), (129, 64), (257, 33),
                                 (1000, 7), (2500, 3), (385, 20)])
def test_fold_unfold(cfa, T, H):
    W = weights(1, H)
    wide = normal(2, T, H * QK + 24)
    q = wide[:, 16:16 + H * QK].unflatten(1, (H, QK))
    o = normal(3, T, H, C)
    q_lat = torch.full((T + 1, H, ROW), 3.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((T + 1, H, V), 3.0, dtype=torch.bfloat16, device="cuda")
    with cfa.Latent(1, 2500, H, 64) as plan:
        plan.fold(q, W, q_lat[:T])
        plan.unfold(o, W, out[:T])
        assert plan.status() == cfa.CFA_OK
    want, size = ref.fold(f64(q), f64(W))
    got = f64(q_lat[:T])
    assert np.all(np.abs(got[..., :C] - want[..., :C]) <= H8 * np.abs(want[..., :C]) + 128 * 2.0 ** -24 * size)
    assert np.array_equal(got[..., C:], want[..., C:])
    want, size = ref.unfold(f64(o), f64(W))
    assert np.all(np.abs(f64(out[:T]) - want) <= H8 * np.abs(want) + 512 * 2.0 ** -24 * size)
    assert torch.all(q_lat[T] == 3.0) and torch.all(out[T] == 3.0)


@pytest.mark.parametrize("T,H", [(20, 3), (300, 40)])
def test_fold_keeps_tokens_and_heads_apart(cfa, T, H):
    """What is not finite in one token's head stays there."""
    W, q, o = weights(1, H), normal(2, T, H, QK), normal(3, T, H, C)
    q[7, 1, 3], o[9, 2, 400] = float("nan"), float("inf")
    q_lat, out = normal(4, T, H, ROW), normal(5, T, H, V)
    with cfa.Latent(1, 512, H, 64) as plan:
        plan.fold(q, W, q_lat)
        plan.unfold(o, W, out)
    for x, at in ((f64(q_lat), (7, 1)), (f64(out), (9, 2))):
        odd = ~np.isfinite(x).all(-1)
        assert odd[at] and odd.sum() == 1


@pytest.mark.parametrize("T,H", [(1, 1024), (20, 1000), (1 << 17, 1)])
def test_fold_unfold_most_heads_and_tokens(cfa, T, H):
    q, o, W = normal(1, T, H, QK), normal(2, T, H, C), weights(3, H)
    with cfa.Latent(1, T, H, 64) as plan:
        ql = plan.fold(q, W, torch.empty(T, H, ROW, dtype=torch.bfloat16, device="cuda"))
        out = plan.unfold(o, W, torch.empty(T, H, V, dtype=torch.bfloat16, device="cuda"))
        assert plan.status() == cfa.CFA_OK
    w = W.double().view(C, H, 256)
    for got, x, m, n, eq in ((ql[..., :C], q[..., :128], w[..., :128], 128, "thd,chd->thc"), (out, o, w[..., 128:], 512, "thc,chd->thd")):
        want, size = torch.einsum(eq, x.double(), m), torch.einsum(eq, x.double().abs(), m.abs())
        assert torch.all((got.double() - want).abs() <= H8 * want.abs() + n * 2.0 ** -24 * size)
    assert same_bits(ql[..., C:], q[..., 128:])


def test_fold_results_past_32_bits(cfa):
    """More than 2^31 values of q_lat: the last tokens are those of a call of their own."""
    T, H, last = 30000, 128, 200
    q, W = normal(1, T, H, QK), weights(2, H)
    with cfa.Latent(1, T, H, 64) as plan:
        far = plan.fold(q, W, torch.empty(T, H, ROW, dtype=torch.bfloat16, device="cuda"))
        near = plan.fold(q[-last:], W, torch.empty(last, H, ROW, dtype=torch.bfloat16, device="cuda"))
        out = plan.unfold(far[..., :C].contiguous(), W, torch.empty(T, H, V, dtype=torch.bfloat16, device="cuda"))
        out2 = plan.unfold(near[..., :C].contiguous(), W, torch.empty(last, H, V, dtype=torch.bfloat16, device="cuda"))
        assert plan.status() == cfa.CFA_OK
    assert same_bits(far[-last:], near) and same_bits(out[-last:], out2)


# ------------------------------------------------- attention over cached rows


def batch(seed, H, ps, lens, news, width=None, lead=0, tail=2, spare=3):
    """A ragged batch; rows that no request holds are NaN, tables past the held pages -1."""
    r = np.random.default_rng(seed)
    held = [-(-L // ps) for L in lens]
    n_pages = sum(held) + spare
    order = r.permutation(n_pages)
    tables = np.full((len(lens), width or max(1, max(held))), -1, dtype=np.int32)
    pages = normal(seed, n_pages, ps, ROW)
    mine = torch.zeros(n_pages, ps, dtype=torch.bool)
    at = 0
    for b, (L, h) in enumerate(zip(lens, held)):
        tables[b, :h] = order[at:at + h]
        for j in range(h):
            mine[order[at + j], :min(ps, L - j * ps)] = True
        at += h
    pages[~mine.cuda()] = float("nan")
    cu = [lead]
    for n in news:
        cu.append(cu[-1] + n)
    T = cu[-1] + tail
    return dict(q=normal(seed + 1, T, H, ROW), cu=cu, lens=list(lens), tables=tables, pages=pages, H=H, T=T)


def attend(cfa, plan, c, scale=None, lse=True, stream=None, out=None):
    out = torch.full((c["T"], c["H"], C), 5.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    z = torch.full((c["T"], c["H"]), 5.0, dtype=torch.float32, device="cuda") if lse else None
    got = plan.attend(c["q"], ints(c["cu"]), ints(c["lens"]), torch.from_numpy(c["tables"]).cuda(), c["pages"],
                      out, scale=scale, lse=z, stream=stream)
    assert got is out
    return out, z


def check_attend(cfa, c, ps, scale=None, plan=None):
    own = plan is None
    plan = plan or cfa.Latent(max(1, len(c["lens"])), max(1, c["T"]), c["H"], ps)
    out, lse = attend(cfa, plan, c, scale)
    assert plan.status() == cfa.CFA_OK
    if own:
        plan.close()
    pages = np.nan_to_num(f64(c["pages"]), nan=0.0)
    want, wl, size = ref.attention(f64(c["q"]), c["cu"], c["lens"], c["tables"], pages, scale)
    a, b = c["cu"][0], c["cu"][-1]
    close(f64(out)[a:b], want[a:b], size[a:b], "out")
    gl = f64(lse)[a:b]
    seen = np.isfinite(wl[a:b])
    assert np.all(np.abs(gl[seen] - wl[a:b][seen]) <= 1e-4) and np.all(gl[~seen] == -math.inf)
    for t, v in ((out, 5.0), (lse, 5.0)):
        assert torch.all(t[:a] == v) and torch.all(t[b:] == v)
    return out, lse


@pytest.mark.parametrize("H,ps,lens,news", [
    (1, 16, [1], [1]),
    (128, 64, [1], [1]),
    (128, 64, [127, 128, 129, 257], [1, 1, 1, 1]),
    (64, 64, [63, 64, 65, 500], [1, 1, 1, 1]),
    (8, 16, [300, 17, 16, 15], [1, 1, 1, 1]),
    (20, 32, [700, 33, 4, 129], [4, 1, 3, 2]),
    (5, 192, [400, 1], [3, 1]),
    (128, 128, [400, 300], [2, 3]),
    (100, 64, [260, 140], [3, 5]),
    (130, 64, [260, 2], [2, 1]),
    (3, 16, [50, 0, 20, 9], [0, 0, 7, 1]),
    (2, 64, [2, 0, 5], [5, 3, 4]),            # tokens that see no row
    (33, 64, [200], [150]),
    (16, 64, [90, 1000, 40], [90, 8, 40]),
])
def test_attend(cfa, H, ps, lens, news):
    check_attend(cfa, batch(len(lens) * 7 + H, H, ps, lens, news), ps)


@pytest.mark.parametrize("H,ps,lens,news", [
    (128, 64, [20000], [1]),                   # one request over the whole GPU
    (128, 64, [9000, 5, 3500, 1], [1, 1, 2, 1]),
    (8, 16, [30000, 100], [1, 1]),
    (32, 64, [int(v) for v in np.random.default_rng(1).integers(1, 700, 200)], [1] * 200),
    (64, 32, [int(v) for v in np.random.default_rng(2).integers(100, 1500, 40)],
     [int(v) for v in np.random.default_rng(3).integers(1, 5, 40)]),
    (2, 16, [int(v) for v in np.random.default_rng(4).integers(0, 40, 1024)], [1] * 1024),
    (128, 64, [1500] * 9, [1] * 9),
])
def test_attend_cut_and_joined(cfa, H, ps, lens, news):
    lens = [max(l, n) if i % 3 else l for i, (l, n) in enumerate(zip(lens, news))]
    check_attend(cfa, batch(len(lens) + H, H, ps, lens, news, lead=1), ps)


def test_attend_scales_and_far_scores(cfa):
    """Scores of hundreds: the maximum moves by far more than a weight's range."""
    c = batch(3, 40, 64, [900, 130], [1, 2])
    c["pages"] *= torch.linspace(0.5, 1.5, c["pages"].shape[0], device="cuda").to(torch.bfloat16)[:, None, None]
    check_attend(cfa, c, 64, scale=1.0 / 192)
    out, lse = attend(cfa, cfa.Latent(2, 8, 40, 64), c, scale=4.0)
    pages = np.nan_to_num(f64(c["pages"]), nan=0.0)
    want, wl, size = ref.attention(f64(c["q"]), c["cu"], c["lens"], c["tables"], pages, 4.0)
    a, b = c["cu"][0], c["cu"][-1]
    # scores up to some 700: 576 fp32 products' error moves a weight by 576 * 2^-24 * 4 sum |q k|, at most 8%
    # of itself; observed as a whole it stays below the size
    assert np.all(np.abs(f64(out)[a:b] - want[a:b]) <= 0.09 * size[a:b] + H8 * np.abs(want[a:b]))
    assert np.all(np.abs(f64(lse)[a:b] - wl[a:b]) <= 0.09)


def test_attend_is_reproducible_and_captured(cfa):
    c = batch(5, 128, 64, [5000, 700, 64], [1, 2, 1])
    with cfa.Latent(3, 16, 128, 64) as plan:
        a, la = attend(cfa, plan, c)
        b, lb = attend(cfa, plan, c)
        assert same_bits(a, b) and torch.equal(la, lb)
        s = torch.cuda.Stream()
        q, cu, lens = c["q"], ints(c["cu"]), ints(c["lens"])
        tables, out, lse = torch.from_numpy(c["tables"]).cuda(), torch.zeros_like(a), torch.zeros_like(la)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            plan.attend(q, cu, lens, tables, c["pages"], out, lse=lse)
        for _ in range(2):
            out.zero_()
            graph.replay()
            assert same_bits(out[:c["cu"][-1]], a[:c["cu"][-1]])
        lens.copy_(ints([100, 700, 10]))  # a recorded call reads lengths anew
        graph.replay()
        torch.cuda.synchronize()
        c2 = dict(c, lens=[100, 700, 10])
        want, _, size = ref.attention(f64(q), c["cu"], c2["lens"], c["tables"], np.nan_to_num(f64(c["pages"])))
        close(f64(out)[:c["cu"][-1]], want[:c["cu"][-1]], size[:c["cu"][-1]])


def test_attend_on_two_streams(cfa):
    c1, c2 = batch(7, 64, 64, [3000, 40], [1, 1]), batch(8, 64, 64, [2500, 90, 1], [2, 1, 1])
    with cfa.Latent(3, 16, 64, 64) as p1, cfa.Latent(3, 16, 64, 64) as p2:
        a, _ = attend(cfa, p1, c1)
        b, _ = attend(cfa, p2, c2)
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(5):
            with torch.cuda.stream(s1):
                x, _ = attend(cfa, p1, c1)
            with torch.cuda.stream(s2):
                y, _ = attend(cfa, p2, c2)
        torch.cuda.synchronize()
        assert same_bits(a, x) and same_bits(b, y)
        assert p1.status() == p2.status() == cfa.CFA_OK


@pytest.mark.parametrize("what", ["descending", "past", "negative"])
def test_attend_refused_offsets(cfa, what):
    c = batch(9, 16, 64, [100, 200], [2, 2])
    c["cu"] = {"descending": [0, 4, 2], "past": [0, 2, c["T"] + 1], "negative": [-1, 2, 4]}[what]
    with cfa.Latent(2, 16, 16, 64) as plan:
        out, lse = attend(cfa, plan, c)
        assert plan.status() == cfa.CFA_ERR_INVALID_ARG
        assert torch.all(out == 5.0) and torch.all(lse == 5.0)
        c["cu"] = [0, 2, 4]
        check_attend(cfa, c, 64, plan=plan)  # the next call is as ever


def test_attend_lengths_and_pages_out_of_range(cfa):
    c = batch(10, 16, 64, [100, 200, 90], [1, 2, 1])
    c["lens"][1] = c["tables"].shape[1] * 64 + 1
    with cfa.Latent(3, 16, 16, 64) as plan:
        out, lse = attend(cfa, plan, c)
        assert plan.status() == cfa.CFA_ERR_INVALID_ARG
        assert not out[1:3].any() and torch.all(lse[1:3] == -math.inf)
        c["lens"][1] = 200
        c["tables"][0, 1], c["tables"][1, 0] = 10 ** 6, -7
        out, lse = attend(cfa, plan, c)
        assert plan.status() == cfa.CFA_ERR_INVALID_ARG
        want, wl, size = ref.attention(f64(c["q"]), c["cu"], c["lens"], c["tables"], np.nan_to_num(f64(c["pages"])))
        close(f64(out)[:4], want[:4], size[:4])
        assert plan.status() == cfa.CFA_OK


@pytest.mark.parametrize("H,n,bad", [(16, 4, float("nan")), (128, 3, float("inf")), (128, 3, float("nan")), (5, 70, float("-inf"))])
def test_attend_rows_not_seen_do_not_show(cfa, H, n, bad):
    """The last new token's row holds what is not finite: tokens before it do not see it."""
    c = batch(11, H, 64, [300, 80], [n, 2])
    with cfa.Latent(2, 256, H, 64) as plan:
        good, gl = attend(cfa, plan, c)
        page = c["tables"][0, 299 // 64]
        c["pages"][page, 299 % 64, 7] = bad
        out, lse = attend(cfa, plan, c)
        assert plan.status() == cfa.CFA_OK
    assert same_bits(out[:n - 1], good[:n - 1]) and torch.equal(lse[:n - 1], gl[:n - 1])
    assert same_bits(out[n:], good[n:])
    # the token that sees it: a score that is NaN or +inf shows everywhere
    x, z = f64(out[n - 1]), f64(c["q"][n - 1, :, 7]) * bad
    hit = np.isnan(z) | (z == math.inf)
    assert np.isnan(x[hit]).all()


def test_attend_shared_pages_many_heads(cfa):
    """Two requests whose tables name the same pages, one page twice; more heads than a tile's rows."""
    c = batch(12, 300, 32, [200, 100], [2, 3])
    c["tables"][1, :3] = c["tables"][0, :3]
    c["tables"][1, 3] = c["tables"][0, 0]
    check_attend(cfa, c, 32)


def test_attend_most_heads(cfa):
    check_attend(cfa, batch(13, 1024, 64, [130, 70], [1, 2]), 64)


def test_pages_past_32_bits(cfa):
    """A cache of more than 2^31 values: rows near its end are written and read."""
    H, ps, n_pages = 20, 64, 60000
    c = batch(14, H, ps, [300, 64, 70], [1, 1, 2], spare=0)
    small, far = c["pages"], torch.zeros(n_pages, ps, ROW, dtype=torch.bfloat16, device="cuda")
    at = np.linspace(0, n_pages - 1, small.shape[0]).astype(np.int64)  # from the first to the last
    far[torch.from_numpy(at).cuda()] = small
    tables = c["tables"].copy()
    tables[tables >= 0] = at[tables[tables >= 0]]
    with cfa.Latent(4, 8, H, ps) as plan:
        a, la = attend(cfa, plan, c)
        b, lb = attend(cfa, plan, dict(c, pages=far, tables=tables))
        assert same_bits(a, b) and torch.equal(la, lb)
        row, g, q = normal(15, 2, ROW), normal(16, C), normal(17, 2, H, QK)
        slots, near = [n_pages * ps - 1, 58300 * ps + 5], torch.zeros(1, ps, ROW, dtype=torch.bfloat16, device="cuda")
        x, y = torch.empty_like(q), torch.empty_like(q)
        plan.append(row, g, q, ints([5, 1 << 20]), ints([3, 4]), near, x)
        plan.append(row, g, q, ints([5, 1 << 20]), ints(slots), far, y)
        assert plan.status() == cfa.CFA_OK
    assert same_bits(far.view(-1, ROW)[slots], near[0, 3:5]) and same_bits(x, y)


def test_attend_without_tokens_in_a_recorded_batch(cfa):
    """A batch recorded for its most requests, replayed with fewer: the others have no tokens."""
    c = batch(18, 64, 64, [900, 70, 64, 5], [1, 1, 1, 1])
    with cfa.Latent(4, 8, 64, 64) as plan:
        out = torch.full((c["T"], 64, C), 5.0, dtype=torch.bfloat16, device="cuda")
        cu, lens, tables = ints(c["cu"]), ints(c["lens"]), torch.from_numpy(c["tables"]).cuda()
        plan.attend(c["q"], cu, lens, tables, c["pages"], out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.attend(c["q"], cu, lens, tables, c["pages"], out)
        for now, new in (([70, 5, 0, 0], [0, 1, 2, 2, 2]), ([0, 0, 0, 0], [0, 0, 0, 0, 0]), (c["lens"], c["cu"])):
            lens.copy_(ints(now))
            cu.copy_(ints(new))
            out.fill_(5.0)
            graph.replay()
            assert plan.status() == cfa.CFA_OK
            want, _, size = ref.attention(f64(c["q"]), new, now, c["tables"], np.nan_to_num(f64(c["pages"])))
            close(f64(out)[:new[-1]], want[:new[-1]], size[:new[-1]])
            assert torch.all(out[new[-1]:] == 5.0)


# ---------------------------------------------------- expanded keys and values


def prompts(seed, H, pairs, lead=0, tail=2):
    """pairs: (new tokens, keys) of each request."""
    cu, ck = [lead], [1]
    for n, L in pairs:
        cu.append(cu[-1] + n)
        ck.append(ck[-1] + L)
    T, S = cu[-1] + tail, ck[-1] + 1
    q = normal(seed, T, H * QK + 16)[:, 8:8 + H * QK].unflatten(1, (H, QK))
    kv = normal(seed + 1, S, H * 256 + 8)[:, :H * 256].unflatten(1, (H, 256))
    k_rope = normal(seed + 2, S, ROW)[:, C:]
    kv[0], kv[-1], k_rope[0], k_rope[-1] = (float("nan"),) * 4
    return dict(q=q, kv=kv, k_rope=k_rope, cu=cu, ck=ck, H=H, T=T, S=S)


def expanded(plan, c, scale=None, lse=True):
    out = torch.full((c["T"], c["H"], V), 5.0, dtype=torch.bfloat16, device="cuda")
    z = torch.full((c["T"], c["H"]), 5.0, dtype=torch.float32, device="cuda") if lse else None
    assert plan.attend_expanded(c["q"], c["kv"], c["k_rope"], ints(c["cu"]), ints(c["ck"]), out, scale=scale,
                                lse=z) is out
    return out, z


@pytest.mark.parametrize("H,pairs", [
    (1, [(1, 1)]),
    (3, [(1, 1), (2, 2), (5, 70)]),
    (2, [(127, 127), (128, 128), (129, 129)]),
    (2, [(255, 255), (257, 300), (1, 513)]),
    (5, [(64, 64), (0, 30), (10, 0), (300, 400)]),   # a request without tokens, one without keys
    (4, [(9, 4), (40, 20)]),                          # tokens that see no key
    (128, [(70, 200)]),
    (1, [(600, 1500)]),
    (2, [(1025, 1025)]),
    (20, [(33, 33)] * 12),
])
def test_expanded(cfa, H, pairs):
    c = prompts(len(pairs) + H, H, pairs, lead=1)
    with cfa.Latent(len(pairs), c["T"], H, 64) as plan:
        out, lse = expanded(plan, c)
        assert plan.status() == cfa.CFA_OK
        out2, _ = expanded(plan, c, lse=False)
        assert same_bits(out, out2)
    want, wl, size = ref.expanded(f64(c["q"]), np.nan_to_num(f64(c["kv"])), np.nan_to_num(f64(c["k_rope"])), c["cu"], c["ck"])
    a, b = c["cu"][0], c["cu"][-1]
    close(f64(out)[a:b], want[a:b], size[a:b])
    gl, seen = f64(lse)[a:b], np.isfinite(wl[a:b])
    assert np.all(np.abs(gl[seen] - wl[a:b][seen]) <= 1e-4) and np.all(gl[~seen] == -math.inf)
    for t in (out, lse):
        assert torch.all(t[:a] == 5.0) and torch.all(t[b:] == 5.0)


@pytest.mark.parametrize("which", ["cu", "ck"])
def test_expanded_refused_offsets(cfa, which):
    c = prompts(3, 4, [(20, 20), (30, 40)])
    for bad in ([0, 60, 50], [0, 20, 10 ** 6], [-1, 20, 50]):
        with cfa.Latent(2, 64, 4, 64) as plan:
            out, lse = expanded(plan, dict(c, **{which: bad}))
            assert plan.status() == cfa.CFA_ERR_INVALID_ARG
            assert torch.all(out == 5.0) and torch.all(lse == 5.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["key", "rope", "value"])
@pytest.mark.parametrize("n,L,j", [(200, 300, 250), (600, 2900, 2500), (600, 2900, 2750)])
def test_expanded_keys_not_seen_do_not_show(cfa, bad, where, n, L, j):
    c = prompts(5, 3, [(n, L), (150, 150)])
    with cfa.Latent(2, 1024, 3, 64) as plan:
        good, gl = expanded(plan, c)
        key, tok = c["ck"][0] + j, n - L + j  # the first token that sees the key
        at = dict(key=c["kv"][key, 1, 5:6], rope=c["k_rope"][key, 9:10], value=c["kv"][key, 1, 128 + 5:128 + 6])[where]
        at.fill_(bad)
        out, lse = expanded(plan, c)
        assert plan.status() == cfa.CFA_OK
    assert same_bits(out[:tok], good[:tok]) and torch.equal(lse[:tok], gl[:tok])
    assert same_bits(out[n:], good[n:])
    if where == "value":
        x = f64(out[tok:n, 1, 5])
        assert (np.isnan(x) if math.isnan(bad) else x == bad).all()
        out[tok:n, 1, 5] = good[tok:n, 1, 5]
        assert same_bits(out, good) and torch.equal(lse, gl)
    else:
        assert same_bits(out[tok:n, 0], good[tok:n, 0]) or where == "rope"


@pytest.mark.parametrize("H,pairs", [
    (3, [(n % 5, n % 7) for n in range(1024)]),                  # the most requests, some without tokens or keys
    (2, [(1 + n % 3, 40 + n) for n in range(300)]),
    (1, [(2500, 2500)]),                                         # tiles that are cut, and joined
    (7, [(130, 2100), (257, 257), (1, 3000), (300, 150)]),
    (3, [(600, 3000), (257, 2700), (800, 2900)]),                # two tiles in a row of a head in a task
    (1, [(2800, 2800), (513, 2561)]),
    (300, [(3, 140)]),
    (20, [(512 - n, 100 + n) for n in range(40)]),               # first halves that see no key, one after another
])
def test_expanded_cut_and_joined(cfa, H, pairs):
    c = prompts(len(pairs) + H, H, pairs, lead=2, tail=130)
    with cfa.Latent(len(pairs), c["T"], H, 64) as plan:
        out, lse = expanded(plan, c)
        assert plan.status() == cfa.CFA_OK
    want, wl, size = ref.expanded(f64(c["q"]), np.nan_to_num(f64(c["kv"])), np.nan_to_num(f64(c["k_rope"])), c["cu"], c["ck"])
    a, b = c["cu"][0], c["cu"][-1]
    close(f64(out)[a:b], want[a:b], size[a:b])
    gl, seen = f64(lse)[a:b], np.isfinite(wl[a:b])
    assert np.all(np.abs(gl[seen] - wl[a:b][seen]) <= 1e-4) and np.all(gl[~seen] == -math.inf)
    for t in (out, lse):
        assert torch.all(t[:a] == 5.0) and torch.all(t[b:] == 5.0)


def test_expanded_scales_and_far_scores(cfa):
    c = prompts(21, 4, [(140, 300), (70, 70)])
    ck, cu = c["ck"], c["cu"]
    with cfa.Latent(2, 256, 4, 64) as plan:
        for scale, slack in ((1.0 / 64, 0.0), (4.0, 0.016)):
            # at scale 4 the error of 192 fp32 products moves a weight by at most 192 * 2^-24 * 4 sum |q k|
            # of itself, 4 sum |q k| being below 650: 0.8%, and the sum of the weights by as much
            out, lse = expanded(plan, c, scale=scale)
            want, wl, size = ref.expanded(f64(c["q"]), np.nan_to_num(f64(c["kv"])), np.nan_to_num(f64(c["k_rope"])), cu, ck, scale)
            a, b = cu[0], cu[-1]
            assert np.all(np.abs(f64(out)[a:b] - want[a:b]) <= H8 * (1.0625 * size[a:b] + np.abs(want[a:b])) + slack * size[a:b])
            assert np.all(np.abs(f64(lse)[a:b] - wl[a:b]) <= 1e-4 + slack)
        assert plan.status() == cfa.CFA_OK


def test_expanded_rows_past_32_bits(cfa):
    """Keys, values and queries whose rows lie more than 2^31 values apart."""
    c = prompts(22, 2, [(90, 200)])
    step, S, T = 11_000_000, c["S"], c["T"]
    wide = torch.empty(S * step + 4096, dtype=torch.bfloat16, device="cuda")
    kv, rope = wide.as_strided((S, 2, 256), (step, 256, 1)), wide.as_strided((S, 64), (step, 1), 1024)
    q = wide.as_strided((T, 2, QK), (step, QK, 1), 2048)
    kv.copy_(c["kv"]), rope.copy_(c["k_rope"]), q.copy_(c["q"])
    with cfa.Latent(1, T, 2, 64) as plan:
        a, la = expanded(plan, c)
        b, lb = expanded(plan, dict(c, kv=kv, k_rope=rope, q=q))
        assert plan.status() == cfa.CFA_OK
    assert same_bits(a, b) and torch.equal(la, lb)


def test_expanded_is_reproducible_and_captured(cfa):
    c = prompts(23, 8, [(300, 900), (65, 65), (1, 700)])
    with cfa.Latent(3, 512, 8, 64) as plan:
        a, la = expanded(plan, c)
        b, lb = expanded(plan, c)
        assert same_bits(a, b) and torch.equal(la, lb)
        cu, ck, out, lse = ints(c["cu"]), ints(c["ck"]), torch.empty_like(a), torch.empty_like(la)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.attend_expanded(c["q"], c["kv"], c["k_rope"], cu, ck, out, lse=lse)
        n = c["cu"][-1]
        for _ in range(3):
            out.zero_()
            graph.replay()
            assert same_bits(out[:n], a[:n]) and torch.equal(lse[:n], la[:n])
        ck.copy_(ints([1, 2, 300, 1000]))  # a recorded call reads offsets anew
        graph.replay()
        assert plan.status() == cfa.CFA_OK
        want, _, size = ref.expanded(f64(c["q"]), np.nan_to_num(f64(c["kv"])), np.nan_to_num(f64(c["k_rope"])), c["cu"], ck.tolist())
        close(f64(out)[:n], want[:n], size[:n])


def test_expanded_on_two_streams(cfa):
    c1, c2 = prompts(24, 16, [(200, 1500)]), prompts(25, 16, [(150, 300), (1, 900), (40, 40)])
    with cfa.Latent(3, 512, 16, 64) as p1, cfa.Latent(3, 512, 16, 64) as p2:
        a, _ = expanded(p1, c1)
        b, _ = expanded(p2, c2)
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(5):
            with torch.cuda.stream(s1):
                x, _ = expanded(p1, c1)
            with torch.cuda.stream(s2):
                y, _ = expanded(p2, c2)
        torch.cuda.synchronize()
        assert same_bits(a, x) and same_bits(b, y)
        assert p1.status() == p2.status() == cfa.CFA_OK


def test_one_plan_serves_its_calls_in_turn(cfa):
    """Both forms, the products and a refused call on one plan, in one stream and without waiting."""
    c, e = batch(26, 16, 64, [2000, 70], [1, 3]), prompts(27, 16, [(150, 900), (20, 20)])
    with cfa.Latent(2, 512, 16, 64) as plan:
        a, _ = attend(cfa, plan, c)
        b, _ = expanded(plan, e)
        assert plan.status() == cfa.CFA_OK
        for _ in range(3):
            bad, _ = attend(cfa, plan, dict(c, cu=[0, 5, 4]))
            x, _ = attend(cfa, plan, c)
            worse, _ = expanded(plan, dict(e, ck=[1, 900, 2]))
            y, _ = expanded(plan, e)
            assert torch.all(bad == 5.0) and torch.all(worse == 5.0)
            assert same_bits(x, a) and same_bits(y, b)
        assert plan.status() == cfa.CFA_ERR_INVALID_ARG
        assert plan.status() == cfa.CFA_OK


# ------------------------------------------------------------- used together


def test_layer_is_its_parts(cfa):
    """One decode step as a server runs it: tables, then the layer; and the parts one by one."""
    H, ps, B = 20, 16, 5
    lens, fresh = [40, 0, 17, 31, 100], [1, 3, 1, 2, 1]
    width = 9
    held = [-(-x // ps) for x in lens]
    r = np.random.default_rng(1)
    ids = r.permutation(40)
    tables = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, h in enumerate(held):
        tables[b, :h] = torch.from_numpy(ids[at:at + h].astype(np.int32))
        at += h
    T = 12  # padded rows
    pages = normal(1, 40, ps, ROW)
    W, g = weights(2, H), normal(3, C)
    a, q = normal(4, T, 64 + ROW)[:, 64:], normal(5, T, H, QK)
    tables, free = tables.cuda(), ints(ids[at:].tolist())
    lens_d, cu, pos, slots = ints(lens), ints([0] * (B + 1)), ints([0] * T), ints([0] * T)
    pool = ints([0, free.numel()])
    with cfa.Paged(B, T, 8, 2, 64, ps) as book, cfa.Latent(B, T, H, ps) as plan:
        plan.set_rope(theta=50000.0, interleaved=True)
        book.build_tables(lens_d, ints(fresh), free, pool, tables, lens_d, pool, cu, pos, slots)
        new = lambda d: torch.full((T, H, d), 2.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        p1, p2 = pages.clone(), pages.clone()
        q1, ql1, o1, out1 = new(QK), new(ROW), new(C), new(V)
        q2, ql2, o2, out2 = new(QK), new(ROW), new(C), new(V)
        lse1, lse2 = torch.zeros(T, H, device="cuda"), torch.zeros(T, H, device="cuda")
        plan.layer(a, g, q, pos, slots, cu, lens_d, tables, p1, W, q1, ql1, o1, out1, eps=1e-5, lse=lse1)
        plan.append(a, g, q, pos, slots, p2, q2, eps=1e-5)
        plan.fold(q2, W, ql2)
        plan.attend(ql2, cu, lens_d, tables, p2, o2, lse=lse2)
        plan.unfold(o2, W, out2)
        assert plan.status() == cfa.CFA_OK and book.status() == cfa.CFA_OK
    n = sum(fresh)
    for x, y in ((p1, p2), (q1, q2), (ql1, ql2), (o1, o2), (out1, out2)):
        assert same_bits(x, y)
    assert torch.equal(lse1, lse2)
    # and against the formulas in 64 bits, from the layer's own rounded intermediates
    f = freqs(dict(theta=50000.0))
    rows = ref.rows(f64(a), f64(g), 1e-5, pos.tolist(), f, True)
    flat = f64(p1).reshape(-1, ROW)
    for t in range(n):
        assert np.all(np.abs(flat[slots[t].item()] - rows[t]) <= H8 * np.abs(rows[t]) + 2.0 ** -16)
    want, _, size = ref.attention(f64(ql1), cu.tolist(), lens_d.tolist(), tables.cpu().numpy(), f64(p1))
    close(f64(o1)[:n], want[:n], size[:n])
    want, size = ref.unfold(f64(o1)[:n], f64(W))
    assert np.all(np.abs(f64(out1)[:n] - want) <= H8 * np.abs(want) + 512 * 2.0 ** -24 * size)


def test_absorbed_and_expanded_forms_agree(cfa):
    """A prompt through both forms: within what their roundings allow of each other."""
    H, ps, n = 4, 64, 150
    W, g = weights(1, H), torch.ones(C, dtype=torch.bfloat16, device="cuda")
    a, q = normal(2, n, ROW), normal(3, n, H, QK)
    pages = torch.zeros(3, ps, ROW, dtype=torch.bfloat16, device="cuda")
    pos = ints(list(range(n)))
    with cfa.Latent(1, n, H, ps) as plan:
        plan.set_rope()
        q_out, q_lat = torch.empty_like(q), torch.empty(n, H, ROW, dtype=torch.bfloat16, device="cuda")
        o_lat, out = torch.empty(n, H, C, dtype=torch.bfloat16, device="cuda"), torch.empty(n, H, V, dtype=torch.bfloat16, device="cuda")
        cu, lens = ints([0, n]), ints([n])
        plan.layer(a, g, q, pos, pos, cu, lens, ints([[0, 1, 2]]), pages, W, q_out, q_lat, o_lat, out)
        rows = pages.view(-1, ROW)[:n]
        kv = (rows[:, :C] @ W).view(n, H, 256)
        out2 = plan.attend_expanded(q_out, kv, rows[:, C:], cu, cu, torch.empty_like(out))
        assert plan.status() == cfa.CFA_OK
    d = (out.float() - out2.float()).norm() / out2.float().norm()
    # roundings in a row: folded queries or keys, weights, o_lat or values, the result: each at most 2^-8 of its
    # size, on scores of size 2 and sums that do not cancel far
    assert d < 6 * H8


def test_decode_loop_recorded_once(cfa):
    """A recorded step grows its requests token by token; the results are those of fresh calls."""
    H, ps, B = 8, 16, 3
    W, g = weights(1, H), normal(2, C)
    a, q = normal(3, B, ROW), normal(4, B, H, QK)
    pages = normal(5, 30, ps, ROW)
    start = [14, 30, 1]
    tables = torch.full((B, 8), -1, dtype=torch.int32)
    ids = list(range(29, -1, -1))
    for b, L in enumerate(start):
        for j in range(-(-L // ps)):
            tables[b, j] = ids.pop()
    with cfa.Paged(B, B, 8, 2, 64, ps) as book, cfa.Latent(B, B, H, ps) as plan:
        plan.set_rope()
        st = dict(lens=ints(start), tables=tables.cuda(), pool=ints([0, len(ids)]), cu=ints([0] * (B + 1)),
                  pos=ints([0] * B), slots=ints([0] * B), pages=pages)
        free, fresh = ints(ids), ints([1] * B)
        buf = [torch.empty(B, H, d, dtype=torch.bfloat16, device="cuda") for d in (QK, ROW, C, V)]

        def step(st, buf):
            book.build_tables(st["lens"], fresh, free, st["pool"], st["tables"], st["lens"], st["pool"], st["cu"],
                              st["pos"], st["slots"])
            plan.layer(a, g, q, st["pos"], st["slots"], st["cu"], st["lens"], st["tables"], st["pages"], W, *buf)

        st2 = {k: v.clone() for k, v in st.items()}
        buf2 = [torch.empty_like(x) for x in buf]
        keep = {k: v.clone() for k, v in st.items()}
        step(st, buf)  # once before the recording
        for k in st:
            st[k].copy_(keep[k])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(st, buf)
        for i in range(20):
            graph.replay()
            step(st2, buf2)
            assert same_bits(buf[3], buf2[3])
        assert st["lens"].tolist() == [x + 20 for x in start] == st2["lens"].tolist()
        assert same_bits(st["pages"], st2["pages"])
        assert plan.status() == cfa.CFA_OK and book.status() == cfa.CFA_OK


# ------------------------------------------------------------------- refusals


def test_binding_refuses(cfa):
    H, ps, T = 4, 64, 3
    pages, q = normal(1, 2, ps, ROW), normal(2, T, H, QK)
    a, g, W = normal(3, T, ROW), normal(4, C), weights(5, H)
    ql, ol = normal(6, T, H, ROW), normal(7, T, H, C)
    pos = ints([0, 1, 2])
    cu, lens, tables = ints([0, T]), ints([T]), ints([[0]])
    with cfa.Latent(1, T, H, ps) as plan:
        with pytest.raises(TypeError):
            plan.append(a.float(), g, q, pos, pos, pages, q)
        with pytest.raises(ValueError):
            plan.append(a[:, 8:], g, q, pos, pos, pages, q)
        with pytest.raises(ValueError):
            plan.append(a, g, q.transpose(0, 1), pos, pos, pages, q)
        with pytest.raises(ValueError):
            plan.append(a, g, q, pos.cpu(), pos, pages, q)
        with pytest.raises(TypeError):
            plan.append(a, g, q, pos.long(), pos, pages, q)
        with pytest.raises(cfa.CfaError):   # more tokens than the plan's
            big = normal(1, T + 1, H, ROW)
            plan.attend(big, ints([0, T + 1]), lens, tables, pages, normal(2, T + 1, H, C))
        with pytest.raises(cfa.CfaError):   # more requests
            plan.attend(ql, ints([0, 1, T]), ints([1, 2]), ints([[0], [1]]), pages, ol)
        with pytest.raises(ValueError):
            plan.attend(ql, cu, lens, tables, normal(1, 2, 32, ROW), ol)
        for scale in (-1.0, 1e-60):
            with pytest.raises(ValueError):
                plan.attend(ql, cu, lens, tables, pages, ol, scale=scale)
        with pytest.raises(cfa.CfaError):
            plan.attend(ql, cu, lens, tables, pages, ol, scale=3e38)
        with pytest.raises(ValueError):
            plan.fold(q, W[:, :-8], ql)
        with pytest.raises(ValueError):
            plan.set_rope(scaling="other")
        assert plan.status() == cfa.CFA_OK


def test_no_tokens(cfa):
    with cfa.Latent(1, 4, 3, 64) as plan:
        e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        plan.append(e(0, ROW), normal(1, C), e(0, 3, QK), ints([]), ints([]), normal(1, 1, 64, ROW), e(0, 3, QK))
        plan.fold(e(0, 3, QK), weights(1, 3), e(0, 3, ROW))
        plan.unfold(e(0, 3, C), weights(1, 3), e(0, 3, V))
        plan.attend(e(0, 3, ROW), ints([0, 0]), ints([5]), ints([[0]]), normal(1, 1, 64, ROW), e(0, 3, C))
        plan.attend_expanded(e(0, 3, QK), e(0, 3, 256), e(0, 64), ints([0, 0]), ints([0, 0]), e(0, 3, V))
        # tokens without any key
        out = plan.attend_expanded(normal(1, 2, 3, QK), e(0, 3, 256), e(0, 64), ints([0, 2]), ints([0, 0]), e(2, 3, V))
        assert not out.any() and plan.status() == cfa.CFA_OK
