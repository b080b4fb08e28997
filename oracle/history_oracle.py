"""fp64 CPU oracle of the user-history attention operators (include/dlrm_history.h), written from
the definitions: loops over tokens and heads in numpy, no code shared with the kernels.

Every function also returns the magnitudes that a tolerance is relative to (the same sums on
absolute values)."""
from __future__ import annotations

import numpy as np


def angles(positions, inv_freq, sections):
    """Angles [N, R/2] in fp64: pair j turns by positions[its axis] * inv_freq[j]."""
    positions = np.atleast_2d(np.asarray(positions, dtype=np.float64))
    inv_freq = np.asarray(inv_freq, dtype=np.float64)
    out, first = [], 0
    for a, many in enumerate(sections):
        for j in range(first, first + many):
            out.append(positions[a] * inv_freq[j])
        first += many
    assert first == len(inv_freq)
    return np.stack(out, 1) if out else np.zeros((positions.shape[1], 0))


def rotate(x, angle, interleaved, back=False):
    """x [N, H, D] with its first 2 * angle.shape[1] elements turned."""
    y = x.copy()
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None] * (-1.0 if back else 1.0)
    half = angle.shape[1]
    ia, ib = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return y


def pair_size(x, pairs, interleaved):
    """|a| + |b| of each element's pair (the element itself where nothing is rotated)."""
    y = np.abs(x)
    ia, ib = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if interleaved else (slice(0, pairs), slice(pairs, 2 * pairs))
    both = y[..., ia] + y[..., ib]
    y[..., ia], y[..., ib] = both, both
    return y


def norm_rope(x, w, angle, interleaved, eps):
    x = np.asarray(x, dtype=np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)
    return rotate(x, angle, interleaved), pair_size(x, angle.shape[1], interleaved)


def norm_rope_bwd(dy, x, w, angle, interleaved, eps):
    """(dx, dw or None, magnitude of dx, magnitude of dw)."""
    g = rotate(np.asarray(dy, dtype=np.float64), angle, interleaved, back=True)
    size = pair_size(np.asarray(dy, dtype=np.float64), angle.shape[1], interleaved)
    if w is None:
        return g, None, size, None
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = x * r
    dx = r * (g * w - u * (g * w * u).mean(-1, keepdims=True))
    mag = r * (size * np.abs(w) + np.abs(u) * (size * np.abs(w * u)).mean(-1, keepdims=True))
    return dx, (g * u).sum((0, 1)), mag, (size * np.abs(u)).sum((0, 1))


def slots(q_offsets, kv_lens, page_table, page, num_pages):
    """(page, slot) of every token, or None for a token that is not stored."""
    out = []
    for s in range(len(kv_lens)):
        m = q_offsets[s + 1] - q_offsets[s]
        for i in range(m):
            at = kv_lens[s] - m + i
            pg = page_table[s][at // page] if 0 <= at < len(page_table[s]) * page else -1
            out.append((int(pg), at % page) if 0 <= pg < num_pages else None)
    return out


def seen(p, held, causal, window):
    """First and past-the-last entry that the token at entry p sees."""
    if not causal:
        return 0, held
    return max(0, p - window + 1) if window else 0, max(0, p + 1)


def attention(q, k_cache, v_cache, q_offsets, kv_lens, page_table, causal, window, scale):
    """out, lse and, per token and head: sum p |v| / l, the largest scale * sum |q||k| and how many
    entries are seen. Entries in pages outside the cache take no part."""
    N, Hq, D = q.shape
    pages, Hk, page, _ = k_cache.shape
    group = Hq // Hk
    out, lse = np.zeros((N, Hq, D)), np.full((N, Hq), -np.inf)
    mag, size, count = np.zeros((N, Hq, D)), np.zeros((N, Hq)), np.zeros((N, Hq), dtype=np.int64)
    for s in range(len(kv_lens)):
        first, last = q_offsets[s], q_offsets[s + 1]
        held = kv_lens[s]
        if last == first or held == 0:
            continue
        entry = np.arange(held)
        where = np.asarray(page_table[s])[entry // page]
        good = (where >= 0) & (where < pages)
        entry, where = entry[good], where[good]
        k = k_cache[where, :, entry % page].astype(np.float64)  # [entries, Hk, D]
        v = v_cache[where, :, entry % page].astype(np.float64)
        for n in range(first, last):
            lo, hi = seen(held - (last - first) + n - first, held, causal, window)
            use = (entry >= lo) & (entry < hi)
            if not use.any():
                continue
            for h in range(Hq):
                kk, vv = k[use, h // group], v[use, h // group]
                z = scale * (kk @ q[n, h].astype(np.float64))
                top = z.max()
                e = np.exp(z - top)
                out[n, h] = e @ vv / e.sum()
                lse[n, h] = top + np.log(e.sum())
                mag[n, h] = e @ np.abs(vv) / e.sum()
                size[n, h] = scale * (np.abs(kk) @ np.abs(q[n, h].astype(np.float64))).max()
                count[n, h] = use.sum()
    return out, lse, mag, size, count
