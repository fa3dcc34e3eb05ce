"""The operators of paged latent caches as measurable cases: the norm, rotation and append
of a token's latent row, the folding of queries into the latent space and of results out of
it, attention over the cached rows (absorbed form), and attention of prompts over expanded
keys and values.

``own = False`` computes each operator from elementary torch operations in 32 bits (64 for
angles); ``own = True`` calls the library through ``out_proj_block_gb300.cfa.Latent``.
"""
import math
import random

import torch

own = False

DEV = "cuda"
C, R, N, V = 512, 64, 128, 128  # latent, rotated, unrotated and value dims
ROW, QK = C + R, N + R          # a cache row; a head's query


# ------------------------------------------------------------------- cases


def listed():
    return [
        # One token of a small model's heads: what the launch costs.
        dict(name="append_t1_h8", op="append", T=1, heads=8, page=64, inter=False, factor=1.0, far=4096),
        # A prompt chunk of the full head count at far positions.
        dict(name="append_t4096_h128", op="append", T=4096, heads=128, page=64, inter=True, factor=40.0,
             far=163840),
        # The queries of a decode step of four requests: the weights bound it.
        dict(name="fold_t4_h128", op="fold", T=4, heads=128),
        # A prompt chunk of odd length.
        dict(name="fold_t777_h32", op="fold", T=777, heads=32),
        # The results of a single request's token.
        dict(name="unfold_t1_h128", op="unfold", T=1, heads=128),
        # A large batch with drafted tokens.
        dict(name="unfold_t1000_h128", op="unfold", T=1000, heads=128),
        # One request of the benchmark's shape: all keys of one row table over the whole GPU.
        dict(name="attend_b1_h128_4k", op="attend", B=1, heads=128, page=64, keys=4096, new=1, lse=False),
        # The serving batch: ragged lengths up to 8192.
        dict(name="attend_b64_h128_8k", op="attend", B=64, heads=128, page=64, keys=8192, new=1, lse=False),
        # Many requests on a share of the heads, small pages.
        dict(name="attend_b200_h32_2k", op="attend", B=200, heads=32, page=32, keys=2048, new=1, lse=False),
        # Verification of up to four drafted tokens a request, odd head count, with the log-sum-exp.
        dict(name="attend_verify_b16_h20", op="attend", B=16, heads=20, page=128, keys=5000, new=4, lse=True),
        # Prompts of a ragged batch from their first token.
        dict(name="expanded_prompts_b5_h32", op="expanded", B=5, heads=32, new=1500, before=0, lse=False),
        # A chunk of one long prompt behind what it has in the cache.
        dict(name="expanded_chunk_h128", op="expanded", B=1, heads=128, new=1024, before=2500, lse=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "fold", "unfold", "attend", "attend", "attend", "expanded", "expanded"])
    heads = rng.choice([8, 20, 32, 64, 128])
    if op == "append":
        return dict(op=op, T=_log(rng, 1, 4096), heads=heads, page=rng.choice([16, 32, 64, 128]),
                    inter=rng.random() < 0.5, factor=rng.choice([1.0, 4.0, 40.0]), far=_log(rng, 64, 163840))
    if op in ("fold", "unfold"):
        return dict(op=op, T=_log(rng, 1, 1000), heads=heads)
    if op == "attend":
        new = rng.choice([1, 1, 1, rng.randint(2, 8)])
        B, keys = _log(rng, 1, 200), _log(rng, max(16, new), 8192)
        while B * keys * max(heads * new, 128) > 64 * 8192 * 128:  # no dearer than the largest listed case
            B = B // 2 if B > 1 else 1
            keys = keys if B > 1 else max(new, keys // 2)
        return dict(op=op, B=B, heads=heads, page=rng.choice([16, 32, 64, 128]), keys=keys, new=new,
                    lse=rng.random() < 0.25)
    B, new, before = _log(rng, 1, 5), _log(rng, 9, 1500), rng.choice([0, 0, _log(rng, 1, 2500)])
    while B * new * (new + before) * heads > 1024 * 3500 * 128:
        new = new * 3 // 4
    return dict(op=op, B=B, heads=heads, new=new, before=before, lse=rng.random() < 0.25)


# ------------------------------------------------------------------ inputs


def _lens(c):
    """Per request (keys, new tokens), the same for every seed (the seed only deals them out)."""
    r = random.Random(str(sorted((k, v) for k, v in c.items() if k != "name")))
    pairs = []
    for _ in range(c["B"]):
        if c["op"] == "attend":
            n = r.randint(1, c["new"])
            pairs.append((r.randint(max(n, c["keys"] // 4), max(n, c["keys"])), n))
        else:
            n = r.randint(max(1, c["new"] // 3), c["new"])
            pairs.append((n + (r.randint(c["before"] // 2, c["before"]) if c["before"] else 0), n))
    if c["op"] == "attend":
        pairs[0] = (max(c["keys"], pairs[0][1]), pairs[0][1])
    else:
        pairs[0] = (c["new"] + c["before"], c["new"])
    return pairs


def _cdiv(a, b):
    return -(-a // b)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)


def _weights(g, heads):
    """W_kvb [512, heads * 256], a head's columns [W_k | W_v], scaled as a trained layer's."""
    w = torch.randn(C, heads * (N + V), generator=g, device=DEV)
    return (w / math.sqrt(C)).to(torch.bfloat16)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _rope_args(c):
    f = c["factor"]
    return dict(theta=10000.0, interleaved=c["inter"], scaling="by_parts" if f > 1.0 else "none", factor=f,
                low_turns=1.0, high_turns=32.0, original_ctx=4096, magnitude=0.1 * math.log(f) + 1.0)


_plans = {}


def _plan(c, seqs, tokens):
    """The library's plan for these sizes, made once, as a serving program keeps it."""
    from out_proj_block_gb300 import cfa
    key = (seqs, tokens, c["heads"], c.get("page", 64), c.get("inter"), c.get("factor"))
    if key not in _plans:
        _plans.clear()
        plan = cfa.Latent(seqs, tokens, c["heads"], key[3])
        if c["op"] == "append":
            plan.set_rope(**_rope_args(c))
        _plans[key] = plan
    return _plans[key]


def prepare(case, seed):
    c = dict(case)
    g = _gen(seed)
    H = c["heads"]
    s = dict(case=c, plan=None)
    if c["op"] == "append":
        T, ps = c["T"], c["page"]
        n_pages = _cdiv(T, ps) + 2
        # the down projection's rows: what the queries are made of, then the latent and the rotated key
        s["a"] = _normal(g, T, 512 + ROW)[:, 512:]
        s["g_kv"] = (1.0 + 0.1 * torch.randn(C, generator=g, device=DEV)).to(torch.bfloat16)
        s["q"] = _normal(g, T, H, QK)
        s["positions"] = torch.randint(0, c["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
        s["slots"] = torch.randperm(n_pages * ps, generator=g, device=DEV)[:T].to(torch.int32)
        s["pages"] = _normal(g, n_pages, ps, ROW)
        s["q_out"] = torch.empty(T, H, QK, dtype=torch.bfloat16, device=DEV)
        s["turns"] = _frequencies(c)
        if own:
            s["plan"] = _plan(c, 1, T)
        return s
    if c["op"] in ("fold", "unfold"):
        T = c["T"]
        s["W_kvb"] = _weights(g, H)
        if c["op"] == "fold":
            s["q"] = _normal(g, T, H, QK)
            s["q_lat"] = torch.empty(T, H, ROW, dtype=torch.bfloat16, device=DEV)
        else:
            s["o_lat"] = _normal(g, T, H, C)
            s["out"] = torch.empty(T, H, V, dtype=torch.bfloat16, device=DEV)
        if own:
            s["plan"] = _plan(c, 1, T)
        return s
    pairs = _lens(c)
    random.Random(seed).shuffle(pairs)
    keys, new = [p[0] for p in pairs], [p[1] for p in pairs]
    T = sum(new)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s.update(cu=_ints(cu), new=new, keys=keys,
             lse=torch.empty(T, H, dtype=torch.float32, device=DEV) if c["lse"] else None)
    if c["op"] == "attend":
        B, ps = c["B"], c["page"]
        held, width = [_cdiv(x, ps) for x in keys], _cdiv(max(keys), ps)
        n_pages = sum(held) + 3
        order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        tables = torch.zeros(B, width, dtype=torch.int32, device=DEV)
        tables[torch.arange(width, device=DEV) < _ints(held)[:, None]] = order[:sum(held)]
        s.update(q_lat=_normal(g, T, H, ROW), pages=_normal(g, n_pages, ps, ROW), tables=tables,
                 lens=_ints(keys), out=torch.empty(T, H, C, dtype=torch.bfloat16, device=DEV))
    else:
        S = sum(keys)
        cu_k = [0]
        for n in keys:
            cu_k.append(cu_k[-1] + n)
        # the rotated keys lie behind the latents they came with
        s.update(q=_normal(g, T, H, QK), kv=_normal(g, S, H, N + V), k_rope=_normal(g, S, ROW)[:, C:],
                 cu_k=_ints(cu_k), out=torch.empty(T, H, V, dtype=torch.bfloat16, device=DEV))
    if own:
        s["plan"] = _plan(c, c["B"], T)
    return s


# --------------------------------------------------------------- the passes


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "fold": _own_fold, "unfold": _own_unfold, "attend": _own_attend,
                "expanded": _own_expanded}[op](state)
    return {"append": _plain_append, "fold": _plain_fold, "unfold": _plain_unfold, "attend": _plain_attend,
            "expanded": _plain_expanded}[op](state)


def _own_append(s):
    s["plan"].append(s["a"], s["g_kv"], s["q"], s["positions"], s["slots"], s["pages"], s["q_out"], eps=1e-6)
    return {"q_out": s["q_out"], "pages": s["pages"]}


def _own_fold(s):
    s["plan"].fold(s["q"], s["W_kvb"], s["q_lat"])
    return s["q_lat"]


def _own_unfold(s):
    s["plan"].unfold(s["o_lat"], s["W_kvb"], s["out"])
    return s["out"]


def _own_attend(s):
    s["plan"].attend(s["q_lat"], s["cu"], s["lens"], s["tables"], s["pages"], s["out"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_expanded(s):
    s["plan"].attend_expanded(s["q"], s["kv"], s["k_rope"], s["cu"], s["cu_k"], s["out"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _frequencies(c):
    """Radians per position of each rotated pair, in 64 bits."""
    r = _rope_args(c)
    i = torch.arange(R // 2, device=DEV, dtype=torch.float64)
    f = r["theta"] ** (-2.0 * i / R)
    if r["scaling"] == "by_parts":
        turns = r["original_ctx"] * f / (2 * math.pi)
        keep = ((turns - r["low_turns"]) / (r["high_turns"] - r["low_turns"])).clamp(0, 1)
        f = f * (keep + (1 - keep) / r["factor"])
    return f


def _plain_rotate(x, cos, sin, inter):
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :R // 2], x[..., R // 2:])
    u, w = a * cos - b * sin, b * cos + a * sin
    return torch.stack((u, w), -1).flatten(-2) if inter else torch.cat((u, w), -1)


def _plain_append(s):
    c = s["case"]
    ang = s["positions"].double()[:, None] * s["turns"]
    m = _rope_args(c)["magnitude"]
    cos, sin = (ang.cos() * m).float(), (ang.sin() * m).float()
    a, q = s["a"].float(), s["q"].float()
    lat = a[:, :C]
    lat = lat * torch.rsqrt(lat.square().mean(-1, keepdim=True) + 1e-6) * s["g_kv"].float()
    row = torch.cat((lat, _plain_rotate(a[:, C:], cos, sin, c["inter"])), -1)
    s["pages"].view(-1, ROW)[s["slots"].long()] = row.to(torch.bfloat16)
    s["q_out"][..., :N] = s["q"][..., :N]
    s["q_out"][..., N:] = _plain_rotate(q[..., N:], cos[:, None], sin[:, None], c["inter"]).to(torch.bfloat16)
    return {"q_out": s["q_out"], "pages": s["pages"]}


def _plain_fold(s):
    T, H = s["q"].shape[:2]
    w = s["W_kvb"].float().view(C, H, N + V)[..., :N].permute(1, 2, 0)  # [H, 128, 512]
    q = s["q"][..., :N].float().transpose(0, 1)                         # [H, T, 128]
    s["q_lat"][..., :C] = torch.matmul(q, w).transpose(0, 1).to(torch.bfloat16)
    s["q_lat"][..., C:] = s["q"][..., N:]
    return s["q_lat"]


def _plain_unfold(s):
    H = s["o_lat"].shape[1]
    w = s["W_kvb"].float().view(C, H, N + V)[..., N:].permute(1, 0, 2)  # [H, 512, 128]
    s["out"].copy_(torch.matmul(s["o_lat"].float().transpose(0, 1), w).transpose(0, 1))
    return s["out"]


def _plain_attend(s):
    c = s["case"]
    B, H, most = c["B"], c["heads"], max(s["new"])
    T = s["q_lat"].shape[0]
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(s["cu"][1:].contiguous(), t.int(), right=True)
    i = t - s["cu"][b]
    q = torch.zeros(B, most, H, ROW, device=DEV)
    q[b, i] = s["q_lat"].float()
    rows = s["pages"][s["tables"].long()].float().flatten(1, 2)  # [B, S, 576]
    S = rows.shape[1]
    x = torch.matmul(q.view(B, most * H, ROW), rows.transpose(1, 2)) / math.sqrt(QK)
    n = s["cu"][1:] - s["cu"][:-1]
    last = (s["lens"] - n)[:, None] + torch.arange(most, device=DEV)  # the last key each query sees
    see = torch.arange(S, device=DEV) <= last[..., None]              # [B, most, S]
    x = x.view(B, most, H, S).masked_fill_(~see[:, :, None], float("-inf"))
    m = x.amax(-1, keepdim=True).clamp_min_(-1e30)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, most * H, S), rows[..., :C]).view(B, most, H, C) / l
    s["out"].copy_(o[b, i])
    if s["lse"] is not None:
        s["lse"].copy_((m + l.log())[b, i, :, 0])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_expanded(s):
    t, k = 0, 0
    for n, L in zip(s["new"], s["keys"]):
        q = s["q"][t:t + n].float().transpose(0, 1)                     # [H, n, 192]
        kn, v = s["kv"][k:k + L].float().transpose(0, 1).split((N, V), -1)
        x = torch.matmul(q[..., :N], kn.transpose(1, 2))
        x += torch.matmul(q[..., N:], s["k_rope"][k:k + L].float().T)
        x *= 1.0 / math.sqrt(QK)
        hide = torch.arange(L, device=DEV) > torch.arange(L - n, L, device=DEV)[:, None]
        x.masked_fill_(hide, float("-inf"))
        m = x.amax(-1, keepdim=True)
        x.sub_(m).exp_()
        l = x.sum(-1, keepdim=True)
        s["out"][t:t + n] = (torch.matmul(x, v) / l).transpose(0, 1).to(torch.bfloat16)
        if s["lse"] is not None:
            s["lse"][t:t + n] = (m + l.log())[..., 0].T
        t, k = t + n, k + L
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- the costs


def work(case):
    c = case
    H = c["heads"]
    if c["op"] == "append":
        return {"bytes": c["T"] * (4 * ROW + 4 * H * QK + 8) + 2 * C, "flops": c["T"] * (4 * C + 3 * R * (H + 1))}
    if c["op"] == "fold":
        return {"bytes": 2 * c["T"] * H * (QK + ROW) + 2 * C * N * H, "flops": 2 * c["T"] * H * N * C}
    if c["op"] == "unfold":
        return {"bytes": 2 * c["T"] * H * (C + V) + 2 * C * V * H, "flops": 2 * c["T"] * H * V * C}
    pairs = _lens(c)
    T, S = sum(n for _, n in pairs), sum(x for x, _ in pairs)
    seen = sum(x - n + i + 1 for x, n in pairs for i in range(n))
    lse = 4 * T * H if c["lse"] else 0
    if c["op"] == "attend":
        return {"bytes": 2 * ROW * S + 2 * T * H * (ROW + C) + lse, "flops": 2 * (ROW + C) * H * seen}
    return {"bytes": 2 * T * H * (QK + V) + 2 * S * (H * (N + V) + R) + lse, "flops": 2 * (QK + V) * H * seen}


# ------------------------------------------------------------ in 64 bits


def exact(case, seed):
    """What run() returns for these inputs, from the definitions in 64 bits, one head, request
    or position at a time."""
    s = prepare(case, seed)
    c = s["case"]
    H = c["heads"]
    if c["op"] == "append":
        half = R // 2
        pair = [(2 * i, 2 * i + 1) if c["inter"] else (i, i + half) for i in range(half)]
        first, second = [p[0] for p in pair], [p[1] for p in pair]
        r = _rope_args(c)
        f = []
        for i in range(half):
            w = math.pow(r["theta"], -2.0 * i / R)
            if c["factor"] > 1.0:
                ramp = (r["original_ctx"] * w / (2 * math.pi) - r["low_turns"]) / (r["high_turns"] - r["low_turns"])
                ramp = min(1.0, max(0.0, ramp))
                w = ramp * w + (1 - ramp) * w / r["factor"]
            f.append(w)
        turn = torch.polar(torch.full((c["T"], half), r["magnitude"], dtype=torch.float64, device=DEV),
                           s["positions"].double()[:, None] * torch.tensor(f, dtype=torch.float64, device=DEV))

        def rotated(x, turn):
            y = x.double().clone()
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            return y

        pages = s["pages"].double()
        lat = s["a"][:, :C].double()
        lat = s["g_kv"].double() * lat / ((lat ** 2).sum(1, keepdim=True) / C + 1e-6).sqrt()
        where = torch.tensor([divmod(x, c["page"]) for x in s["slots"].tolist()], device=DEV)
        pages[where[:, 0], where[:, 1], :C] = lat
        pages[where[:, 0], where[:, 1], C:] = rotated(s["a"][:, C:], turn)
        q = s["q"].double()
        q[..., N:] = rotated(s["q"][..., N:], turn[:, None])
        return {"q_out": q, "pages": pages}
    if c["op"] in ("fold", "unfold"):
        W = s["W_kvb"].double()
        out = torch.empty(c["T"], H, ROW if c["op"] == "fold" else V, dtype=torch.float64, device=DEV)
        for h in range(H):
            at = h * (N + V)
            if c["op"] == "fold":
                out[:, h, :C] = s["q"][:, h, :N].double() @ W[:, at:at + N].T
                out[:, h, C:] = s["q"][:, h, N:].double()
            else:
                out[:, h] = s["o_lat"][:, h].double() @ W[:, at + N:at + N + V]
        return out
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(out.shape[:2], dtype=torch.float64, device=DEV)
    cu = s["cu"].tolist()
    k0 = 0
    for b in range(c["B"]):
        n, L = s["new"][b], s["keys"][b]
        hide = torch.arange(L, device=DEV)[None] > (L - n + torch.arange(n, device=DEV))[:, None]
        if c["op"] == "attend":
            at = torch.arange(L, device=DEV)
            rows = s["pages"][s["tables"][b].long()[at // c["page"]], at % c["page"]].double()
            for i in range(n):
                q = s["q_lat"][cu[b] + i].double()
                x = (q @ rows.T / math.sqrt(QK)).masked_fill(hide[i], float("-inf"))
                z = torch.logsumexp(x, 1)
                out[cu[b] + i] = torch.exp(x - z[:, None]) @ rows[:, :C]
                lse[cu[b] + i] = z
        else:
            for h in range(H):
                q = s["q"][cu[b]:cu[b + 1], h].double()
                k = torch.cat((s["kv"][k0:k0 + L, h, :N], s["k_rope"][k0:k0 + L]), 1).double()
                x = (q @ k.T / math.sqrt(QK)).masked_fill(hide, float("-inf"))
                z = torch.logsumexp(x, 1)
                out[cu[b]:cu[b + 1], h] = torch.exp(x - z[:, None]) @ s["kv"][k0:k0 + L, h, N:].double()
                lse[cu[b]:cu[b + 1], h] = z
        k0 += L
    return {"out": out, "lse": lse if c["lse"] else None}
