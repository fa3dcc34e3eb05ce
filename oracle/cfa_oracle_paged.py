"""fp64 reference of the paged-cache operators, from their definitions: plain
loops over requests, tokens and heads with numpy, no code of the library.
Used by the tests only."""
from __future__ import annotations

import math

import numpy as np


def build_tables(lens, fresh, free_pages, pool, tables, base, page_size, n_slots):
    """The step's tables and maps, or the refused form; integers throughout.
    Returns (granted, tables, lens_out, pool_out, cu, positions, slots)."""
    B, width = tables.shape
    tables = tables.copy()
    positions, slots = [0] * n_slots, [-1] * n_slots
    ok = all(l >= 0 and f >= 0 and l + f <= width * page_size for l, f in zip(lens, fresh))
    ok = ok and sum(fresh) <= n_slots
    takes = [math.ceil((l + f) / page_size) - math.ceil(l / page_size) for l, f in zip(lens, fresh)]
    ok = ok and sum(takes) <= min(pool[1], len(free_pages)) - pool[0]
    if not ok:
        return False, tables, list(lens), list(pool), [0] * (B + 1), positions, slots
    taken, cu = pool[0], [0]
    for b in range(B):
        have = math.ceil(lens[b] / page_size)
        for j in range(takes[b]):
            tables[b, have + j] = free_pages[taken]
            taken += 1
        for i in range(fresh[b]):
            at = lens[b] + i
            positions[cu[b] + i] = base + at
            slots[cu[b] + i] = int(tables[b, at // page_size]) * page_size + at % page_size
        cu.append(cu[b] + fresh[b])
    return True, tables, [l + f for l, f in zip(lens, fresh)], [taken, pool[1]], cu, positions, slots


def frequencies(theta, rotary_dim, scaling="none", factor=1.0, low_turns=1.0, high_turns=32.0,
                original_ctx=4096):
    """Radians per position of every pair."""
    f = []
    for i in range(rotary_dim // 2):
        w = theta ** (-2.0 * i / rotary_dim)
        if scaling == "linear":
            w = w / factor
        elif scaling == "by_parts":
            r = original_ctx * w / (2.0 * math.pi)
            g = min(1.0, max(0.0, (r - low_turns) / (high_turns - low_turns)))
            w = g * w + (1.0 - g) * w / factor
        f.append(w)
    return f


def rotate(x, positions, freqs, interleaved=False, magnitude=1.0):
    """x [T, heads, d] float64 -> rotated copy."""
    y = np.array(x, dtype=np.float64)
    half = len(freqs)
    for t, n in enumerate(positions):
        for i, f in enumerate(freqs):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = magnitude * math.cos(n * f), magnitude * math.sin(n * f)
            y[t, :, a] = c * x[t, :, a] - s * x[t, :, b]
            y[t, :, b] = c * x[t, :, b] + s * x[t, :, a]
    return y


def cache_rows(pages, table, n, head, page_size):
    """The first n rows of one head behind a page table, [n, d] float64; a page
    id outside the cache reads as zeros."""
    d = pages.shape[-1]
    out = np.zeros((n, d))
    for j in range(n):
        page = int(table[j // page_size])
        if 0 <= page < pages.shape[0]:
            out[j] = pages[page, head, j % page_size]
    return out


def attention(q, cu, lens, tables, k_pages, v_pages, prefix_table=(), prefix_len=0, scale=None):
    """out [T, heads, d] and lse [T, heads] in float64, and the mean magnitude
    sum_j w_j |v_j| / sum_j w_j that bounds how roundings of the weights show;
    rows outside the requests are NaN."""
    T, H, d = q.shape
    kv, ps = k_pages.shape[1], k_pages.shape[2]
    G = H // kv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = np.full((T, H, d), np.nan)
    size = np.full((T, H, d), np.nan)
    lse = np.full((T, H), np.nan)
    for g in range(kv):
        Kp = cache_rows(k_pages, prefix_table, prefix_len, g, ps)
        Vp = cache_rows(v_pages, prefix_table, prefix_len, g, ps)
        for b in range(len(lens)):
            n, L = cu[b + 1] - cu[b], lens[b]
            K = np.concatenate((Kp, cache_rows(k_pages, tables[b], L, g, ps)))
            V = np.concatenate((Vp, cache_rows(v_pages, tables[b], L, g, ps)))
            for i in range(n):
                see = prefix_len + min(L, max(0, L - n + i + 1))
                t = cu[b] + i
                for h in range(g * G, (g + 1) * G):
                    if see == 0:
                        out[t, h], size[t, h], lse[t, h] = 0.0, 0.0, -math.inf
                        continue
                    s = scale * (K[:see] @ q[t, h])
                    m = s.max()
                    w = np.exp(s - m)
                    out[t, h] = w @ V[:see] / w.sum()
                    size[t, h] = w @ np.abs(V[:see]) / w.sum()
                    lse[t, h] = m + math.log(w.sum())
    return out, lse, size
