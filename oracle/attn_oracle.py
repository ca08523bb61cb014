"""fp64 CPU definitions of the softmax attention calls (numpy): rotary positions, the
8-bit form of a cached head, attention of one sequence with what bounds its rounding
errors, and reading sequences out of a paged cache. Test infrastructure only, like the
rest of this package."""

from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def rotate(x, positions, cos_sin, interleaved=False):
    """x [T, H, D]: the first rot channels turned by the table's rows [cos | sin]."""
    rot = cos_sin.shape[1]
    half = rot // 2
    c, s = cos_sin[positions][:, None, :half], cos_sin[positions][:, None, half:]
    first = np.arange(half) * 2 if interleaved else np.arange(half)
    second = first + (1 if interleaved else half)
    y = np.array(x, np.float64)
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


def power_scale(x):
    """The smallest power of two s with max |x| <= 448 s over the last axis; 1 for zeros."""
    m = np.max(np.abs(x), axis=-1)
    safe = np.where(m > 0, m, 1.0)
    s = 2.0 ** np.ceil(np.log2(safe / E4M3_MAX))
    s = np.where(safe > E4M3_MAX * s, 2 * s, s)  # (log2 may round a value just above a power to it)
    return np.where(m > 0, np.maximum(s, 2.0 ** -110), 1.0)


def attend(q, k, v, scale, seen):
    """One sequence: q [T, HQ, D], k and v [S, HKV, D], seen [T] keys that each query sees
    (the first ones). Returns (o, lse, a, top): a [T, HQ, D] is sum_j p_ij |v_j|, and top
    [T, HQ] the largest sum of |q||k| scale of a key that the row sees."""
    T, HQ, D = q.shape
    HKV = k.shape[1]
    G = HQ // HKV
    o, a = np.zeros((T, HQ, v.shape[2])), np.zeros((T, HQ, v.shape[2]))
    lse, top = np.full((T, HQ), -np.inf), np.zeros((T, HQ))
    for h in range(HQ):
        kh, vh = k[:, h // G], v[:, h // G]
        for i in range(T):
            n = int(seen[i])
            if n <= 0:
                continue
            s = kh[:n] @ q[i, h] * scale
            top[i, h] = np.max(np.abs(kh[:n]) @ np.abs(q[i, h])) * scale
            m = np.max(s)
            e = np.exp(s - m)
            lse[i, h] = m + np.log(e.sum())
            p = e / e.sum()
            o[i, h], a[i, h] = p @ vh[:n], p @ np.abs(vh[:n])
    return o, lse, a, top


def seen_keys(T, S, causal):
    """How many keys each of T queries on S keys sees."""
    return np.clip(np.arange(T) + S - T + 1, 0, S) if causal else np.full(T, S)


def tokens_of(cache, table, n, scale=None):
    """The first n tokens on the pages of table: cache [pages, HKV, P, D] -> [n, HKV, D]."""
    P = cache.shape[2]
    x = np.zeros((n, cache.shape[1], cache.shape[3]))
    for j in range(n):
        page = int(table[j // P])
        x[j] = cache[page, :, j % P]
        if scale is not None:
            x[j] *= scale[page, :, j % P, None]
    return x
