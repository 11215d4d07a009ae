"""Plain 64-bit restatement of the attention beside the indexer: the rotated
append into the paged key/value cache and the decode attention that reads it.

Loops over tokens, rows and heads, straight from the formulas; caches are
numpy arrays [pages, 64, heads, dim].
"""

from __future__ import annotations

import numpy as np

PAGE = 64


def rotate(x, angles_cos, angles_sin, interleaved):
    """x [heads, dim] of one token, its first 2 * len(cos) columns turned pair by pair."""
    out = np.array(x, dtype=np.float64)
    half = len(angles_cos)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = float(angles_cos[i]), float(angles_sin[i])
        out[:, a] = x[:, a] * c - x[:, b] * s
        out[:, b] = x[:, b] * c + x[:, a] * s
    return out


def append(k, v, slots, k_cache, v_cache, positions=None, cos_sin=None, q=None, interleaved=False):
    """Writes k', v into k_cache, v_cache (in place) and returns q' (or None)."""
    q_out = None if q is None else np.array(q, dtype=np.float64)
    for i, slot in enumerate(slots):
        kk = np.asarray(k[i], dtype=np.float64)
        if cos_sin is not None:
            p = min(max(int(positions[i]), 0), len(cos_sin) - 1)
            half = cos_sin.shape[1] // 2
            c, s = cos_sin[p, :half], cos_sin[p, half:]
            kk = rotate(kk, c, s, interleaved)
            if q is not None:
                q_out[i] = rotate(np.asarray(q[i], dtype=np.float64), c, s, interleaved)
        if 0 <= slot < k_cache.shape[0] * PAGE:
            k_cache[slot // PAGE, slot % PAGE] = kk
            v_cache[slot // PAGE, slot % PAGE] = v[i]
    return q_out


def request_of(row, starts):
    """The request that holds a row, or None for a padding row."""
    for j in range(len(starts) - 1):
        if starts[j] <= row < starts[j + 1]:
            return j
    return None


def visible(row, starts, row_ends, block_table, prefix_pages=(), prefix_len=0, topk=None):
    """(page, token) of every key the row sees, in order."""
    j = request_of(row, starts)
    if j is None:
        return []
    if topk is not None:
        own = [int(t) for t in topk[row] if 0 <= t < row_ends[row]]
    else:
        own = range(int(row_ends[row]))
    keys = [(int(prefix_pages[t // PAGE]), t % PAGE) for t in range(prefix_len)]
    return keys + [(int(block_table[j][t // PAGE]), t % PAGE) for t in own]


def attend(q, k_cache, v_cache, keys, scale):
    """One row: q [heads, dim] over the (page, token) list.  Returns the output,
    the log-sum-exp, the weighted mean of |v| and the largest sum |q||k| scale
    (the two magnitudes that rounding errors scale with)."""
    heads, dim = q.shape
    hkv = k_cache.shape[2]
    if not keys:
        return np.zeros((heads, dim)), np.full(heads, -np.inf), np.zeros((heads, dim)), np.zeros(heads)
    pages = np.array([p for p, _ in keys])
    toks = np.array([t for _, t in keys])
    k = np.asarray(k_cache[pages, toks], dtype=np.float64)     # [n, hkv, dim]
    v = np.asarray(v_cache[pages, toks], dtype=np.float64)
    of = np.arange(heads) // (heads // hkv)
    qd = np.asarray(q, dtype=np.float64)
    s = np.empty((heads, len(keys)))
    size = np.empty(heads)
    out = np.empty((heads, dim))
    mean_abs = np.empty((heads, dim))
    lse = np.empty(heads)
    for h in range(heads):
        s[h] = k[:, of[h]] @ qd[h] * scale
        size[h] = (np.abs(k[:, of[h]]) @ np.abs(qd[h])).max() * scale
        top = s[h].max()
        w = np.exp(s[h] - top)
        lse[h] = top + np.log(w.sum())
        w = w / w.sum()
        out[h] = w @ v[:, of[h]]
        mean_abs[h] = w @ np.abs(v[:, of[h]])
    return out, lse, mean_abs, size
