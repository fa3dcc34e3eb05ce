"""What the paged-cache operators do on the GPU with device data out of range: refused or
skipped as a whole, flagged in the status word, and nothing else changed."""
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


@pytest.mark.parametrize("B,T,each,prefix", [(64, 32, 32, 0), (64, 32, 32, 100), (600, 100, 3, 70)])
def test_attention_offsets_up_and_down(cfa, B, T, each, prefix):
    """Every second request looks right by itself, and together they count the same tokens many
    times over: refused, with no row touched. The plan has room for all that are counted."""
    nh, nkv, d, ps = 8, 2, 64, 64
    pages = 8
    cu = [each * (b % 2) for b in range(B + 1)]
    q, kp, vp = normal(1, T, nh, d), normal(2, pages, nkv, ps, d), normal(3, pages, nkv, ps, d)
    out = torch.full((T, nh, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, nh), 7.0, device="cuda")
    lens, tables = ints([40] * B), torch.zeros(B, 2, dtype=torch.int32, device="cuda")
    good = ints([min(b, T) for b in range(B + 1)])
    kw = dict(prefix_table=ints([1, 2]), prefix_len=prefix) if prefix else {}
    with cfa.Paged(B, 4096, nh, nkv, d, ps) as plan:
        for _ in range(2):
            plan.attend(q, ints(cu), lens, tables, kp, vp, out, lse=lse, **kw)
            assert torch.all(out == 7.0) and torch.all(lse == 7.0)
            assert plan.status() == cfa.CFA_ERR_INVALID_ARG
        first, again = torch.empty_like(out), torch.empty_like(out)
        plan.attend(q, good, lens, tables, kp, vp, first, lse=lse, **kw)
        plan.attend(q, ints(cu), lens, tables, kp, vp, out, **kw)
        assert plan.status() == cfa.CFA_ERR_INVALID_ARG
        plan.attend(q, good, lens, tables, kp, vp, again, lse=lse, **kw)
        n = min(B, T)
        assert torch.equal(first[:n], again[:n]) and torch.all(out == 7.0)
        assert plan.status() == cfa.CFA_OK


@pytest.mark.parametrize("pool", [[1, -1], [0, -(1 << 31)], [(1 << 31) - 1, -2], [-2, (1 << 31) - 1], [-3, -2]])
@pytest.mark.parametrize("fresh", [[5, 0, 9], [1, 0, 0]])
def test_tables_pool_counters_below_zero(cfa, pool, fresh):
    """Refused whole, also where no page is wanted."""
    lens, tables, n = [16, 4, 30], [[3, -7, -7], [2, -7, -7], [4, 5, -7]], 20
    if fresh[0] == 1:
        lens = [15, 4, 30]
    t, new_lens, new_pool = ints(tables), ints([-9] * 3), ints([-9] * 2)
    cu, pos, slots = ints([-9] * 4), ints([-9] * n), ints([-9] * n)
    with cfa.Paged(3, 32, 8, 2, 64, 16) as plan:
        plan.build_tables(ints(lens), ints(fresh), ints([9, 8, 7]), ints(pool), t, new_lens, new_pool, cu, pos, slots)
        assert plan.status() == cfa.CFA_ERR_INVALID_ARG
        assert t.tolist() == tables and new_lens.tolist() == lens and new_pool.tolist() == pool
        assert cu.tolist() == [0] * 4 and pos.tolist() == [0] * n and slots.tolist() == [-1] * n
        good = ints([0, 3])
        plan.build_tables(ints(lens), ints(fresh), ints([9, 8, 7]), good, t, new_lens, good, cu, pos, slots)
        assert plan.status() == cfa.CFA_OK
        assert new_lens.tolist() == [a + b for a, b in zip(lens, fresh)] and cu.tolist()[-1] == sum(fresh)


@pytest.mark.parametrize("over", ["cu", "lens", "tables", "prefix_table"])
def test_layer_refuses_writing_over_what_it_reads(cfa, over):
    T, nh, nkv, d, ps = 4, 4, 2, 64, 16
    q, k, v = normal(1, T, nh, d), normal(2, T, nkv, d), normal(3, T, nkv, d)
    kp, vp, q_out, out = normal(4, 8, nkv, ps, d), normal(5, 8, nkv, ps, d), normal(6, T, nh, d), normal(7, T, nh, d)
    a = dict(q=q, k=k, v=v, positions=ints([5] * T), slots=ints([16, 17, 32, 48]), cu=ints([0, 2, 3, 4]),
             lens=ints([2, 1, 1]), tables=ints([[1], [2], [3]]), k_pages=kp, v_pages=vp, q_out=q_out, out=out,
             prefix_table=ints([5]), prefix_len=9)
    with cfa.Paged(3, T, nh, nkv, d, ps) as plan:
        plan.layer(**a)
        assert plan.status() == cfa.CFA_OK
        before = [x.clone() for x in (kp, vp, q_out, out)]
        for t in (kp, vp, q_out, out):
            there = t.view(-1).view(torch.int32)[8:8 + a[over].numel()].view(a[over].shape)
            with pytest.raises(cfa.CfaError):
                plan.layer(**{**a, over: there})
        assert all(torch.equal(x, y) for x, y in zip(before, (kp, vp, q_out, out)))
        assert plan.status() == cfa.CFA_OK


def test_a_new_plan_behind_a_busy_default_stream(cfa):
    """The plan's words are zero when create returns, and stay what later kernels make them, for
    streams that do not wait for the default one too."""
    side = torch.cuda.Stream()
    lens, fresh, n = ints([0] * 5), ints([300] * 5), 2048
    tables = torch.full((5, 20), -1, dtype=torch.int32, device="cuda")
    free, pool, cu = ints(range(100)), ints([0, 100]), ints([0] * 6)
    pos, slots = ints([0] * n), ints([0] * n)
    torch.cuda.synchronize()
    for turn in range(4):
        torch.cuda._sleep(200_000_000)
        with cfa.Paged(5, n, 8, 2, 64, 16) as plan:
            with torch.cuda.stream(side):
                lens.zero_()
                pool.copy_(ints([0, 100] if turn % 2 else [0, 90]))
                plan.build_tables(lens, fresh, free, pool, tables, lens, pool, cu, pos, slots)
                side.synchronize()
                assert lens.tolist() == ([300] * 5 if turn % 2 else [0] * 5)
                assert plan.status() == (cfa.CFA_OK if turn % 2 else cfa.CFA_ERR_NO_PAGES)


def test_scales_that_32_bits_do_not_hold(cfa):
    """A scale that rounds to 0 would be taken as the default, one near the largest number
    becomes infinite when it is turned to base 2. The smallest one makes the mean of the values."""
    nh, d, n = 2, 64, 40
    q, kp, vp = normal(1, 1, nh, d), normal(2, 1, nh, 64, d), normal(3, 1, nh, 64, d)
    out, lse = torch.empty_like(q), torch.empty(1, nh, device="cuda")
    a = dict(q=q, cu=ints([0, 1]), lens=ints([n]), tables=ints([[0]]), k_pages=kp, v_pages=vp, out=out, lse=lse)
    with cfa.Paged(1, 1, nh, nh, d, 64) as plan:
        for scale, error in ((1e-50, ValueError), (5e-324, ValueError), (3e38, cfa.CfaError), (1e39, cfa.CfaError)):
            with pytest.raises(error):
                plan.attend(**a, scale=scale)
        plan.attend(**a, scale=1e-45)
        assert plan.status() == cfa.CFA_OK
    want = vp[0, :, :n].double().mean(1)
    # 40 weights of one, exact in bf16: only the result is rounded
    assert torch.all((out[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6)
    assert torch.all((lse.double() - torch.log(torch.tensor(float(n)))).abs() <= 1e-5)


@pytest.mark.parametrize("n,own,prefix", [(32768, 40, 9), (16384, 16384, 0)])
def test_attention_of_some_hundred_thousand_tiles(cfa, n, own, prefix):
    """1024 query heads on one key head: tiles of a quarter of a token. A few rows against 64
    bits (as in the other attention tests: the weights and the result rounded to bf16)."""
    nh, d, ps = 1024, 64, 64
    pages = 1 + -(-own // ps)
    kp, vp = normal(1, pages, 1, ps, d), normal(2, pages, 1, ps, d)
    q = torch.empty(n, nh, d, dtype=torch.bfloat16, device="cuda")
    q.copy_(normal(3, 64, nh, d).repeat(n // 64, 1, 1))
    out, lse = torch.full_like(q, 7.0), torch.empty(n, nh, device="cuda")
    kw = dict(prefix_table=ints([0]), prefix_len=prefix) if prefix else {}
    with cfa.Paged(1, n, nh, 1, d, ps) as plan:
        plan.attend(q, ints([0, n]), ints([own]), ints([list(range(1, pages))]), kp, vp, out, lse=lse, **kw)
        assert plan.status() == cfa.CFA_OK
    for i in (0, 1, n // 3, n - own, n - 1):
        see = max(0, own - n + i + 1)
        k, v = (torch.cat((x[0, 0, :prefix], x[1:, 0].reshape(-1, d)[:see])).double() for x in (kp, vp))
        for h in (0, 255, 256, 1023):
            s = k @ q[i, h].double() / 8.0
            w = torch.softmax(s, 0)
            want, size = w @ v, w @ v.abs()
            tol = (1 + 2.0 ** -4) * 2.0 ** -8 * (want.abs() + size) + 1e-6
            assert torch.all((out[i, h].double() - want).abs() <= tol)
            assert abs(float(lse[i, h]) - float(torch.logsumexp(s, 0))) <= 1e-4
    assert torch.all(torch.isfinite(out.view(-1)[:: 997]))
