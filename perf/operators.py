"""The paged-cache operators as measurable cases: block tables and slot maps from request
lengths, rotary embedding with the append to the cache, and attention of a ragged batch
over a shared prefix and its own pages.

``own = False`` computes each operator from elementary torch operations in 32 bits (64 for
angles); ``own = True`` calls the library through ``out_proj_block_gb300.cfa.Paged``.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases


def listed():
    return [
        # One decode step's bookkeeping of a small batch: one new token per request.
        dict(name="tables_decode_b16", op="tables", B=16, page=16, cached=4096, chunk=1, chunks=0),
        # Bookkeeping of a full mixed batch: one request in eight brings a prompt chunk.
        dict(name="tables_mixed_b512", op="tables", B=512, page=64, cached=6784, chunk=2048, chunks=64),
        # The new tokens of a decode step, 32 heads x 128, half layout over the whole head.
        dict(name="append_decode_b16", op="append", T=16, heads=32, kv=32, d=128, page=16,
             rd=128, inter=False, scaling="none", factor=1.0, far=4096),
        # A prompt chunk with shared key heads, rotated by parts for a long context, half the head.
        dict(name="append_chunk_t4096", op="append", T=4096, heads=32, kv=8, d=128, page=64,
             rd=64, inter=True, scaling="by_parts", factor=8.0, far=131072),
        # An odd number of tokens, 64 heads x 64, interpolated positions.
        dict(name="append_d64_t777", op="append", T=777, heads=64, kv=64, d=64, page=32,
             rd=64, inter=False, scaling="linear", factor=4.0, far=16384),
        # The smallest call: one request, a short prompt.
        dict(name="attend_b1", op="attend", B=1, heads=32, kv=32, d=128, page=64, prefix=64,
             own=64, new=1, chunk=False, lse=False),
        # The decode batch of the fused block's shape behind a common system prompt.
        dict(name="attend_mha_b16", op="attend", B=16, heads=32, kv=32, d=128, page=64, prefix=4096,
             own=1024, new=1, chunk=False, lse=False),
        # A large batch that asks about one long document.
        dict(name="attend_gqa_b64_p32k", op="attend", B=64, heads=32, kv=8, d=128, page=64,
             prefix=32768, own=2048, new=1, chunk=False, lse=False),
        # Many short requests behind a common prompt: the products bound it, not the cache.
        dict(name="attend_gqa_b256_p8k", op="attend", B=256, heads=32, kv=8, d=128, page=16,
             prefix=8192, own=512, new=1, chunk=False, lse=False),
        # 64 heads x 64, small batch.
        dict(name="attend_d64_b8", op="attend", B=8, heads=64, kv=64, d=64, page=128, prefix=2048,
             own=2048, new=1, chunk=False, lse=False),
        # Verification of up to 8 drafted tokens a request, odd prefix, with the log-sum-exp.
        dict(name="attend_verify_b32", op="attend", B=32, heads=32, kv=8, d=128, page=32,
             prefix=12345, own=700, new=8, chunk=False, lse=True),
        # Prompt chunks of a ragged batch behind the prefix.
        dict(name="attend_chunks_b8", op="attend", B=8, heads=32, kv=8, d=128, page=64, prefix=4096,
             own=1500, new=512, chunk=True, lse=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "append", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    if op == "tables":
        B = _log(rng, 1, 512)
        return dict(op=op, B=B, page=page, cached=_log(rng, 16, 6784), chunk=_log(rng, 1, 2048),
                    chunks=rng.randint(0, max(0, min(64, B))))
    heads, kv, d = rng.choice([(32, 32, 128), (32, 8, 128), (64, 64, 64), (64, 8, 128), (28, 4, 128),
                               (16, 2, 64), (40, 8, 64)])
    if op == "append":
        scaling = rng.choice(["none", "linear", "by_parts"])
        return dict(op=op, T=_log(rng, 1, 4096), heads=heads, kv=kv, d=d, page=page,
                    rd=rng.choice([d, d // 2]), inter=rng.random() < 0.5, scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                    far=_log(rng, 64, 131072))
    kind = rng.choice(["decode", "decode", "verify", "chunk"])
    if kind == "decode":
        B, new, prefix, mine = _log(rng, 1, 256), 1, _log(rng, 1, 32768), _log(rng, 1, 2048)
    elif kind == "verify":
        B, new, prefix, mine = _log(rng, 1, 32), rng.randint(2, 8), _log(rng, 1, 16384), _log(rng, 8, 1024)
    else:
        B, new, prefix, mine = _log(rng, 1, 8), _log(rng, 9, 160), _log(rng, 1, 4096), _log(rng, 160, 1500)
    # products and cache stay below the largest listed cases'
    while B * new * prefix * heads * d > 64 * 32768 * 4096:
        prefix //= 2
    while (prefix + B * mine) * kv * d > 80000 * 1024:
        mine, prefix = (mine // 2, prefix) if B * mine > prefix else (mine, prefix // 2)
    mine = max(mine, new)
    return dict(op=op, B=B, heads=heads, kv=kv, d=d, page=page, prefix=prefix, own=mine, new=new,
                chunk=kind == "chunk", lse=rng.random() < 0.25)


# ------------------------------------------------------------------ inputs


def _lens(c):
    """The case's request lengths, the same for every seed (the seed only deals them out):
    tables -> (cached, fresh) pairs; attend -> (own length, new tokens) pairs."""
    r = random.Random(str(sorted((k, v) for k, v in c.items() if k != "name")))
    if c["op"] == "tables":
        pairs = [(r.randint(0, c["cached"]), 1) for _ in range(c["B"])]
        for i in range(c["chunks"]):
            pairs[i] = (pairs[i][0], r.randint(1, c["chunk"]))
        return pairs
    pairs = []
    for _ in range(c["B"]):
        n = r.randint(max(1, c["new"] // 2 if c["chunk"] else 1), c["new"])
        pairs.append((r.randint(min(c["own"], n + c["own"] // 16), c["own"]), n))
    pairs[0] = (c["own"], pairs[0][1])
    return pairs


def _cdiv(a, b):
    return -(-a // b)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


_plans = {}


def _plan(c, seqs, tokens):
    """The library's plan for these sizes, made once, as a serving program keeps it."""
    from out_proj_block_gb300 import cfa
    key = (seqs, tokens, c.get("heads", 32), c.get("kv", 8), c.get("d", 128), c["page"],
           c.get("rd"), c.get("inter"), c.get("scaling"), c.get("factor"))
    if key not in _plans:
        _plans.clear()
        plan = cfa.Paged(seqs, tokens, key[2], key[3], key[4], key[5])
        if c["op"] == "append":
            plan.set_rope(**_rope_args(c))
        _plans[key] = plan
    return _plans[key]


def _rope_args(c):
    return dict(theta=10000.0, rotary_dim=c["rd"], interleaved=c["inter"], scaling=c["scaling"],
                factor=c["factor"], low_turns=1.0, high_turns=32.0, original_ctx=4096,
                magnitude=0.1 * math.log(c["factor"]) + 1.0)


def prepare(case, seed):
    c = dict(case)
    g = _gen(seed)
    deal = random.Random(seed)
    s = dict(case=c, plan=None)
    if c["op"] == "append":
        T, d, ps = c["T"], c["d"], c["page"]
        n_pages = _cdiv(T, ps) + 2
        # q, k and v as a fused projection leaves them: one row per token
        qkv = _normal(g, T, (c["heads"] + 2 * c["kv"]) * d)
        nq, nk = c["heads"] * d, c["kv"] * d
        s["q"] = qkv[:, :nq].unflatten(1, (c["heads"], d))
        s["k"] = qkv[:, nq:nq + nk].unflatten(1, (c["kv"], d))
        s["v"] = qkv[:, nq + nk:].unflatten(1, (c["kv"], d))
        s["positions"] = torch.randint(0, c["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
        s["slots"] = torch.randperm(n_pages * ps, generator=g, device=DEV)[:T].to(torch.int32)
        s["k_pages"] = _normal(g, n_pages, c["kv"], ps, d)
        s["v_pages"] = _normal(g, n_pages, c["kv"], ps, d)
        s["q_out"] = torch.empty(T, c["heads"], d, dtype=torch.bfloat16, device=DEV)
        s["turns"] = _frequencies(c)
        if own:
            s["plan"] = _plan(c, 1, T)
        return s
    pairs = _lens(c)
    deal.shuffle(pairs)
    B, ps = c["B"], c["page"]
    if c["op"] == "tables":
        cached, fresh = [p[0] for p in pairs], [p[1] for p in pairs]
        width = _cdiv(c["cached"] + max(c["chunk"], 1), ps) + 1
        held = [_cdiv(x, ps) for x in cached]
        need = sum(_cdiv(x + f, ps) - h for x, f, h in zip(cached, fresh, held))
        order = torch.randperm(sum(held) + need + 7, generator=g, device=DEV).to(torch.int32)
        tables = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        h = _ints(held)
        col = torch.arange(width, device=DEV)
        tables[col < h[:, None]] = order[:sum(held)]
        T = _cdiv(sum(fresh), 64) * 64  # the token buffers are padded, as a recorded graph's are
        s.update(lens=_ints(cached), fresh=_ints(fresh), tables=tables,
                 free=order[sum(held):].contiguous(), pool=_ints([3, need + 7]),
                 base=c["page"] * 4, lens_out=torch.empty(B, dtype=torch.int32, device=DEV),
                 pool_out=torch.empty(2, dtype=torch.int32, device=DEV),
                 cu=torch.empty(B + 1, dtype=torch.int32, device=DEV),
                 positions=torch.empty(T, dtype=torch.int32, device=DEV),
                 slots=torch.empty(T, dtype=torch.int32, device=DEV))
        if own:
            s["plan"] = _plan(c, B, T)
        return s
    mine, new = [p[0] for p in pairs], [p[1] for p in pairs]
    P, d = c["prefix"], c["d"]
    n_prefix, width = _cdiv(P, ps), _cdiv(max(mine), ps)
    held = [_cdiv(x, ps) for x in mine]
    n_pages = n_prefix + sum(held) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    tables = torch.zeros(B, width, dtype=torch.int32, device=DEV)
    tables[torch.arange(width, device=DEV) < _ints(held)[:, None]] = order[n_prefix:n_prefix + sum(held)]
    T = sum(new)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s.update(q=_normal(g, T, c["heads"], d), k_pages=_normal(g, n_pages, c["kv"], ps, d),
             v_pages=_normal(g, n_pages, c["kv"], ps, d), prefix_table=order[:n_prefix].contiguous(),
             prefix_len=P, tables=tables, lens=_ints(mine), cu=_ints(cu), most=max(new),
             out=torch.empty(T, c["heads"], d, dtype=torch.bfloat16, device=DEV),
             lse=torch.empty(T, c["heads"], dtype=torch.float32, device=DEV) if c["lse"] else None)
    if own:
        s["plan"] = _plan(c, B, T)
    return s


# --------------------------------------------------------------- the passes


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tables": _own_tables, "append": _own_append, "attend": _own_attend}[op](state)
    return {"tables": _plain_tables, "append": _plain_append, "attend": _plain_attend}[op](state)


def _own_tables(s):
    s["plan"].build_tables(s["lens"], s["fresh"], s["free"], s["pool"], s["tables"], s["lens_out"],
                           s["pool_out"], s["cu"], s["positions"], s["slots"], base=s["base"])
    return {k: s[k] for k in ("tables", "lens_out", "pool_out", "cu", "positions", "slots")}


def _own_append(s):
    s["plan"].append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_pages"], s["v_pages"],
                     s["q_out"])
    return {k: s[k] for k in ("q_out", "k_pages", "v_pages")}


def _own_attend(s):
    s["plan"].attend(s["q"], s["cu"], s["lens"], s["tables"], s["k_pages"], s["v_pages"], s["out"],
                     prefix_table=s["prefix_table"], prefix_len=s["prefix_len"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_tables(s):
    ps = s["case"]["page"]
    lens, fresh, tables, slots = s["lens"].long(), s["fresh"].long(), s["tables"], s["slots"]
    have, need = (lens + ps - 1) // ps, (lens + fresh + ps - 1) // ps
    took = (need - have).cumsum(0)
    rank = took - (need - have)
    s["cu"][:1] = 0
    s["cu"][1:] = fresh.cumsum(0)
    s["lens_out"].copy_(lens + fresh)
    s["pool_out"].copy_(s["pool"])
    s["pool_out"][:1] += took[-1:].int()
    col = torch.arange(tables.shape[1], device=DEV)
    at = s["pool"][0] + rank[:, None] + (col - have[:, None])
    got = s["free"][at.clamp(0, s["free"].numel() - 1)]
    tables.copy_(torch.where((col >= have[:, None]) & (col < need[:, None]), got, tables))
    t = torch.arange(slots.numel(), device=DEV)
    live = t < s["cu"][-1]
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True).clamp(max=lens.numel() - 1)
    pos = torch.where(live, lens[b] + t - s["cu"][b], 0)
    s["positions"].copy_(torch.where(live, pos + s["base"], 0))
    s["slots"].copy_(torch.where(live, tables[b, pos // ps].long() * ps + pos % ps, -1))
    return {k: s[k] for k in ("tables", "lens_out", "pool_out", "cu", "positions", "slots")}


def _frequencies(c):
    """Radians per position of each rotated pair, in 64 bits."""
    r = _rope_args(c)
    i = torch.arange(c["rd"] // 2, device=DEV, dtype=torch.float64)
    f = r["theta"] ** (-2.0 * i / c["rd"])
    if r["scaling"] == "linear":
        f = f / r["factor"]
    if r["scaling"] == "by_parts":
        turns = r["original_ctx"] * f / (2 * math.pi)
        keep = ((turns - r["low_turns"]) / (r["high_turns"] - r["low_turns"])).clamp(0, 1)
        f = f * (keep + (1 - keep) / r["factor"])
    return f


def _plain_rotate(x, cos, sin, rd, inter):
    x = x.float()
    a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if inter else (x[..., :rd // 2], x[..., rd // 2:rd])
    u, w = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((u, w), -1).flatten(-2) if inter else torch.cat((u, w), -1)
    return torch.cat((y, x[..., rd:]), -1).to(torch.bfloat16)


def _plain_append(s):
    c = s["case"]
    ang = s["positions"].double()[:, None] * s["turns"]
    m = _rope_args(c)["magnitude"]
    cos, sin = (ang.cos() * m).float()[:, None], (ang.sin() * m).float()[:, None]
    s["q_out"].copy_(_plain_rotate(s["q"], cos, sin, c["rd"], c["inter"]))
    k = _plain_rotate(s["k"], cos, sin, c["rd"], c["inter"])
    page, at = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
    s["k_pages"][page, :, at] = k
    s["v_pages"][page, :, at] = s["v"]
    return {k: s[k] for k in ("q_out", "k_pages", "v_pages")}


def _rows_of(pages, table, n):
    """The first n cache rows of a list of pages, in 32 bits: [kv, n, d]."""
    x = pages[table.long()].float()  # [m, kv, ps, d]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _plain_attend(s):
    c = s["case"]
    T, kv, d, G = s["q"].shape[0], c["kv"], c["d"], c["heads"] // c["kv"]
    B, most, P = c["B"], s["most"], s["prefix_len"]
    scale = 1.0 / math.sqrt(d)
    q = s["q"].float().view(T, kv, G, d)
    # the prefix: every token's rows against the same keys
    K, V = _rows_of(s["k_pages"], s["prefix_table"], P), _rows_of(s["v_pages"], s["prefix_table"], P)
    x = torch.matmul(q.transpose(0, 1).reshape(kv, T * G, d), K.transpose(1, 2)) * scale
    m1 = x.amax(-1, keepdim=True)
    x.sub_(m1).exp_()
    l1, o1 = x.sum(-1, keepdim=True), torch.matmul(x, V)
    del x
    back = lambda t: t.reshape(kv, T, G, -1).transpose(0, 1)  # noqa: E731  -> [T, kv, G, *]
    m1, l1, o1 = back(m1), back(l1), back(o1)
    # the requests' own rows: queries padded to the most new tokens of a request
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(s["cu"][1:].contiguous(), t.int(), right=True)
    i = t - s["cu"][b]
    qp = torch.zeros(B, most, kv, G, d, device=DEV)
    qp[b, i] = q
    S = s["tables"].shape[1] * c["page"]
    Ks = s["k_pages"][s["tables"].long()].float().permute(0, 2, 1, 3, 4).reshape(B, kv, S, d)
    x = torch.matmul(qp.permute(0, 2, 1, 3, 4).reshape(B, kv, most * G, d), Ks.transpose(2, 3)) * scale
    del Ks
    n = s["cu"][1:] - s["cu"][:-1]
    last = (s["lens"] - n)[:, None] + torch.arange(most, device=DEV)  # the last key each query sees
    see = torch.arange(S, device=DEV) <= last[..., None]              # [B, most, S]
    x = x.view(B, kv, most, G, S).masked_fill_(~see[:, None, :, None, :], float("-inf"))
    m2 = x.amax(-1, keepdim=True)
    x.sub_(m2).exp_()
    l2 = x.sum(-1, keepdim=True)
    Vs = s["v_pages"][s["tables"].long()].float().permute(0, 2, 1, 3, 4).reshape(B, kv, S, d)
    o2 = torch.matmul(x.view(B, kv, most * G, S), Vs).view(B, kv, most, G, d)
    del x, Vs
    m2, l2, o2 = m2[b, :, i], l2[b, :, i], o2[b, :, i]                # [T, kv, G, *]
    m = torch.maximum(m1, m2)
    w1, w2 = (m1 - m).exp(), (m2 - m).exp()
    l = l1 * w1 + l2 * w2
    s["out"].copy_(((o1 * w1 + o2 * w2) / l).reshape(T, kv * G, d))
    if s["lse"] is not None:
        s["lse"].copy_((m + l.log()).reshape(T, kv * G))
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- the costs


def work(case):
    c = case
    if c["op"] == "tables":
        pairs, ps = _lens(c), c["page"]
        T = sum(f for _, f in pairs)
        taken = sum(_cdiv(x + f, ps) - _cdiv(x, ps) for x, f in pairs)
        # lengths in, lengths and offsets out; positions and slots; free pages to the tables,
        # and the last held page of each request that goes on in it
        return {"bytes": 16 * c["B"] + 8 * T + 8 * taken + 4 * sum(x % ps > 0 for x, _ in pairs) + 16,
                "flops": 0}
    if c["op"] == "append":
        rows = c["T"] * (c["heads"] + 2 * c["kv"])
        return {"bytes": 4 * rows * c["d"] + 8 * c["T"],
                "flops": 3 * c["T"] * (c["heads"] + c["kv"]) * c["rd"]}
    pairs = _lens(c)
    T = sum(n for _, n in pairs)
    seen = sum(c["prefix"] + x - n + i + 1 for x, n in pairs for i in range(n))
    kept = c["prefix"] + sum(x for x, _ in pairs)
    return {"bytes": 4 * c["d"] * c["kv"] * kept + 4 * T * c["heads"] * c["d"] + (4 * T * c["heads"] if c["lse"] else 0),
            "flops": 4 * c["d"] * c["heads"] * seen}


# ------------------------------------------------------------ in 64 bits


def exact(case, seed):
    """What run() returns for these inputs, from the definitions in 64 bits, one request and
    one position at a time. The tables are whole numbers and have no such value."""
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "append":
        half = c["rd"] // 2
        pair = [(2 * i, 2 * i + 1) if c["inter"] else (i, i + half) for i in range(half)]
        first, second = [p[0] for p in pair], [p[1] for p in pair]
        r = _rope_args(c)
        f = []
        for i in range(half):
            w = math.pow(r["theta"], -2.0 * i / c["rd"])
            if r["scaling"] == "linear":
                w /= r["factor"]
            elif r["scaling"] == "by_parts":
                ramp = (r["original_ctx"] * w / (2 * math.pi) - r["low_turns"]) / (r["high_turns"] - r["low_turns"])
                ramp = min(1.0, max(0.0, ramp))
                w = ramp * w + (1 - ramp) * w / r["factor"]
            f.append(w)
        turn = torch.polar(torch.full((c["T"], half), r["magnitude"], dtype=torch.float64, device=DEV),
                           s["positions"].double()[:, None] * torch.tensor(f, dtype=torch.float64, device=DEV))

        def rotated(x):
            y = x.double()
            z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
            y[..., first], y[..., second] = z.real, z.imag
            return y

        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        slot = s["slots"].tolist()
        k, v = rotated(s["k"]), s["v"].double()
        where = torch.tensor([divmod(x, c["page"]) for x in slot], device=DEV)
        kp[where[:, 0], :, where[:, 1]] = k
        vp[where[:, 0], :, where[:, 1]] = v
        return {"q_out": rotated(s["q"]), "k_pages": kp, "v_pages": vp}
    G, ps, P = c["heads"] // c["kv"], c["page"], c["prefix"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    lens, cu = s["lens"].tolist(), s["cu"].tolist()

    def rows(pages, table, n, h):
        at = torch.arange(n, device=DEV)
        return pages[table.long()[at // ps], h, at % ps].double()

    for h in range(c["kv"]):
        Kp, Vp = rows(s["k_pages"], s["prefix_table"], P, h), rows(s["v_pages"], s["prefix_table"], P, h)
        for b in range(c["B"]):
            n, L = cu[b + 1] - cu[b], lens[b]
            q = s["q"][cu[b]:cu[b + 1], h * G:(h + 1) * G].double().reshape(n * G, -1)
            K, V = rows(s["k_pages"], s["tables"][b], L, h), rows(s["v_pages"], s["tables"][b], L, h)
            x = torch.cat((q @ Kp.T, q @ K.T), 1) / math.sqrt(c["d"])
            i = torch.arange(n, device=DEV).repeat_interleave(G)
            hide = torch.arange(P + L, device=DEV)[None] > (P + L - n + i)[:, None]
            x[hide] = float("-inf")
            z = torch.logsumexp(x, 1)
            p = torch.exp(x - z[:, None])
            out[cu[b]:cu[b + 1], h * G:(h + 1) * G] = (p[:, :P] @ Vp + p[:, P:] @ V).view(n, G, -1)
            lse[cu[b]:cu[b + 1], h * G:(h + 1) * G] = z.view(n, G)
    return {"out": out, "lse": lse if c["lse"] else None}
