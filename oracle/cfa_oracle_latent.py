"""fp64 reference of the paged latent-cache operators, from their definitions: plain
loops over requests and tokens with numpy, no code of the library. Used by the tests only."""
from __future__ import annotations

import math

import numpy as np

from oracle import cfa_oracle_paged

C, R, N, V = 512, 64, 128, 128


def rows(a, g, eps, positions, freqs, interleaved=False, magnitude=1.0):
    """Cache rows [T, 576] of down-projection rows a; freqs None: no rotation."""
    lat, rot = a[:, :C], a[:, C:]
    lat = g * lat / np.sqrt((lat ** 2).mean(1, keepdims=True) + eps)
    if freqs is not None:
        rot = cfa_oracle_paged.rotate(rot[:, None], positions, freqs, interleaved, magnitude)[:, 0]
    return np.concatenate((lat, rot), 1)


def queries(q, positions, freqs, interleaved=False, magnitude=1.0):
    """Queries [T, H, 192] with their last 64 dims rotated."""
    if freqs is None:
        return q.copy()
    rot = cfa_oracle_paged.rotate(q[:, :, N:], positions, freqs, interleaved, magnitude)
    return np.concatenate((q[:, :, :N], rot), 2)


def fold(q, W):
    """[T, H, 576], and the sums of magnitudes of the first 512."""
    H = q.shape[1]
    w = W.reshape(C, H, N + V)[:, :, :N]
    lat = np.einsum("thd,chd->thc", q[:, :, :N], w, optimize=True)
    size = np.einsum("thd,chd->thc", np.abs(q[:, :, :N]), np.abs(w), optimize=True)
    return np.concatenate((lat, q[:, :, N:]), 2), size


def unfold(o, W):
    """[T, H, 128], and the sums of magnitudes."""
    H = o.shape[1]
    w = W.reshape(C, H, N + V)[:, :, N:]
    return (np.einsum("thc,chd->thd", o, w, optimize=True),
            np.einsum("thc,chd->thd", np.abs(o), np.abs(w), optimize=True))


def _softmax_sum(q, k, v, scale):
    """q [H, d], k [n, d] or [n, H, d], v likewise -> out [H, dv], lse [H], size [H, dv]."""
    H = q.shape[0]
    if len(k) == 0:
        z = np.zeros((H, v.shape[-1]))
        return z, np.full(H, -math.inf), z
    if k.ndim == 2:
        s = scale * (q @ k.T)
    else:
        s = scale * np.einsum("hd,nhd->hn", q, k, optimize=True)
    m = s.max(1, keepdims=True)
    w = np.exp(s - m)
    l = w.sum(1, keepdims=True)
    if v.ndim == 2:
        o, size = w @ v, w @ np.abs(v)
    else:
        o, size = (np.einsum("hn,nhd->hd", w, x, optimize=True) for x in (v, np.abs(v)))
    return o / l, (m + np.log(l))[:, 0], size / l


def attention(q, cu, lens, tables, pages, scale=None):
    """out [T, H, 512], lse [T, H], and sum_j w_j |row_j| / sum_j w_j, which bounds how roundings of
    the weights show; tokens outside the requests are NaN."""
    T, H, _ = q.shape
    ps = pages.shape[1]
    scale = 1.0 / math.sqrt(N + R) if scale is None else scale
    out, size = np.full((T, H, C), np.nan), np.full((T, H, C), np.nan)
    lse = np.full((T, H), np.nan)
    for b, L in enumerate(lens):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        r = cfa_oracle_paged.cache_rows(pages[:, None], tables[b], L, 0, ps)
        for i in range(n):
            see = max(0, L - n + i + 1)
            t = cu[b] + i
            out[t], lse[t], size[t] = _softmax_sum(q[t], r[:see], r[:see, :C], scale)
    return out, lse, size


def expanded(q, kv, k_rope, cu, cu_k, scale=None):
    """out [T, H, 128], lse [T, H], size as in attention."""
    T, H, _ = q.shape
    scale = 1.0 / math.sqrt(N + R) if scale is None else scale
    out, size = np.full((T, H, V), np.nan), np.full((T, H, V), np.nan)
    lse = np.full((T, H), np.nan)
    for b in range(len(cu) - 1):
        n, L, k0 = cu[b + 1] - cu[b], cu_k[b + 1] - cu_k[b], cu_k[b]
        for i in range(n):
            see = max(0, L - n + i + 1)
            t = cu[b] + i
            k = np.concatenate((kv[k0:k0 + see, :, :N], np.broadcast_to(k_rope[k0:k0 + see, None], (see, H, R))), 2)
            out[t], lse[t], size[t] = _softmax_sum(q[t], k, kv[k0:k0 + see, :, N:], scale)
    return out, lse, size
