"""Plain references of rotary positions, the rotated append, block selection and
block-sparse attention: numpy in 64 bits, written from the formulas that
``include/pa.h`` states, with no code shared with the kernels."""
from __future__ import annotations

import numpy as np


def rotary(x, positions, cos_sin, pair_axis=None, interleaved=False):
    """Rows x [T, H, D] turned; positions [T] or [axes, T].  Returns (values, magnitudes),
    float64: what each element is, and the sum of the absolute values it is made of."""
    y = np.array(x, dtype=np.float64)
    mag = np.abs(y)
    pos = np.asarray(positions).reshape(-1, y.shape[0])
    half = cos_sin.shape[1] // 2
    for t in range(y.shape[0]):
        for i in range(half):
            row = cos_sin[pos[pair_axis[i] if pair_axis is not None else 0, t]].astype(np.float64)
            c, s = row[i], row[half + i]
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
            p, q = y[t, :, a].copy(), y[t, :, b].copy()
            y[t, :, a], y[t, :, b] = p * c - q * s, q * c + p * s
            mag[t, :, a], mag[t, :, b] = abs(p * c) + abs(q * s), abs(q * c) + abs(p * s)
    return y, mag


def bounds_of(keys):
    """(least, largest) of the keys [n, H, D] of a block, NaN where one is."""
    return np.min(keys, axis=0), np.max(keys, axis=0)  # numpy's min and max hand a NaN on


def scores(q, lo, hi):
    """Score of each block: q [G, D], lo, hi [blocks, D] -> [blocks]."""
    q, lo, hi = (np.asarray(x, dtype=np.float64) for x in (q, lo, hi))
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.einsum("gd,bd->gb", np.maximum(q, 0), hi) + np.einsum("gd,bd->gb", np.minimum(q, 0), lo)
    return np.max(s, axis=0)


def query_positions(seqlens_k, cu=None):
    """(request, last visible position) of each packed query."""
    if cu is None:
        return [(r, int(n) - 1) for r, n in enumerate(seqlens_k)]
    return [(r, int(seqlens_k[r]) - int(cu[r + 1] - cu[r]) + i)
            for r in range(len(seqlens_k)) for i in range(int(cu[r + 1] - cu[r]))]


def choose(score, visible, top_k, first, last):
    """top_k of blocks 0..visible-1, ascending, -1 behind them."""
    out = np.full(top_k, -1, dtype=np.int32)
    if visible <= top_k:
        out[:visible] = np.arange(visible)
        return out
    forced = list(range(first)) + list(range(visible - last, visible))
    rank = sorted(range(first, visible - last), key=lambda j: (not np.isnan(score[j]), -score[j], j))
    out[:] = sorted(forced + rank[:top_k - first - last])
    return out


def select(q, bounds, table, seqlens_k, top_k, bs, first=1, last=1, cu=None):
    """selected [Tq, Hkv, top_k] of q [Tq, Hq, D], bounds [NB, Hkv, 2, D]."""
    hkv = bounds.shape[1]
    rows = query_positions(seqlens_k, cu)
    out = np.full((q.shape[0], hkv, top_k), -1, dtype=np.int32)
    g = q.shape[1] // hkv
    for t, (r, pos) in enumerate(rows):
        if pos < 0:
            continue
        n = pos // bs + 1
        for h in range(hkv):
            b = bounds[table[r, :n], h]
            out[t, h] = choose(scores(q[t, h * g:(h + 1) * g], b[:, 0], b[:, 1]), n, top_k, first, last)
    return out


def attend(q, k_cache, v_cache, table, seqlens_k, selected, scale, cu=None):
    """Outputs [Tq, Hq, D], and of each (query, kv head) what its error depends on:
    the largest sum of |q||k| of a visible position (times scale), the largest |v|, the
    number of positions; float64."""
    tq, hq, d = q.shape
    bs, hkv = k_cache.shape[1], k_cache.shape[2]
    g = hq // hkv
    out = np.zeros((tq, hq, d))
    info = np.zeros((tq, hkv, 3))
    for t, (r, pos) in enumerate(query_positions(seqlens_k, cu)):
        for h in range(hkv):
            at = [(int(j), o) for j in selected[t, h] if j >= 0 for o in range(bs) if int(j) * bs + o <= pos]
            if not at:
                continue
            k = np.array([k_cache[table[r, j], o, h] for j, o in at], dtype=np.float64)
            v = np.array([v_cache[table[r, j], o, h] for j, o in at], dtype=np.float64)
            x = q[t, h * g:(h + 1) * g].astype(np.float64)
            s = x @ k.T * scale
            with np.errstate(invalid="ignore"):
                w = np.exp(s - s.max(1, keepdims=True))
                out[t, h * g:(h + 1) * g] = (w @ v) / w.sum(1, keepdims=True)
                info[t, h] = scale * (np.abs(x) @ np.abs(k).T).max(), np.abs(v).max(), len(at)
    return out, info
