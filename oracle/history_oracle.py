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


def pages_assign(new, users, held, tables, free, count, page, n, out_width):
    """Pages handed out one by one. Returns (refusal bits, outputs, state): q_offsets, kv_lens, page_table, slots and
    positions, and held, tables and count after the call, all as lists; refused calls change nothing."""
    U, width = len(held), len(tables[0]) if len(tables) else 0
    held, tables = list(held), [list(r) for r in tables]
    valid = [0 <= u < U for u in users]
    fits = [v and 0 <= held[u] <= width * page for u, v in zip(users, valid)]
    before = [held[u] if f else 0 for u, f in zip(users, fits)]
    grown = [max(m, 0) for m in new]
    pages = lambda e: -(-e // page)
    bits = 0
    if not all(valid):
        bits |= 16
    if any(v and not f for v, f in zip(valid, fits)) or any(m < 0 for m in new) or sum(grown) > n:
        bits |= 2
    if not 0 <= count <= len(free):
        bits |= 4
    need = sum(pages(h + m) - pages(h) if v else pages(m) for h, m, v in zip(before, grown, valid))
    if any(h + m > out_width * page for h, m in zip(before, grown)) or need > count:
        bits |= 8
    if not bits and len({u for u, m in zip(users, new) if m > 0}) < sum(m > 0 for m in new):
        bits |= 16
    slots, positions, offsets, lens, rows = [], [], [0], [], []
    stack, refused = list(free[:max(count, 0)]), bits != 0
    for u, h, m in zip(users, before, grown):
        if refused:
            m = 0
        for i in range(pages(h), pages(h + m)):
            tables[u][i] = stack.pop()
        row = list(tables[u][:min(pages(h + m), out_width)]) if h + m else []
        rows.append(row + [-1] * (out_width - len(row)))
        for e in range(h, h + m):
            p = tables[u][e // page]
            good = 0 <= p < len(free)
            bits |= 0 if good else 4
            slots.append(p * page + e % page if good else -1)
            positions.append(e)
        offsets.append(offsets[-1] + m)
        lens.append(h + m)
        if m:
            held[u] = h + m
    rest = [-1] * (n - len(slots))
    return bits, (offsets, lens, rows, slots + rest, positions + rest), (held, tables, len(stack) if count >= 0 else count)


def pages_release(users, keep, held, tables, free, count, page):
    """(refusal bits, held, free list, count) after the release."""
    U, width = len(held), len(tables[0]) if len(tables) else 0
    held, free = list(held), list(free)
    valid = [0 <= u < U for u in users]
    bits = 0 if all(valid) else 16
    if any(v and not 0 <= held[u] <= width * page for u, v in zip(users, valid)) or any(k < 0 for k in keep):
        bits |= 2
    pages = lambda e: -(-e // page)
    moved = []
    for u, k, v in zip(users, keep, valid):
        h = held[u] if v and 0 <= held[u] <= width * page else 0
        moved.append((u, pages(min(max(k, 0), h)), pages(h), min(max(k, 0), h)))
    if not 0 <= count <= len(free) or count + sum(b - a for _, a, b, _ in moved) > len(free):
        bits |= 4
    if not bits and len(set(users)) < len(users):
        bits |= 16
    if not bits and any(not 0 <= p < len(free) for u, a, b, _ in moved for p in tables[u][a:b]):
        bits |= 4
    if bits:
        return bits, held, free, count
    for u, a, b, k in moved:
        free[count:count + b - a] = tables[u][a:b]
        count += b - a
        held[u] = k
    return 0, held, free, count


def e4m3_values():
    """What the 256 codes stand for: sign, 4 bits of exponent with bias 7, 3 of significand; 0x7f and 0xff are NaN."""
    out = np.empty(256)
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        x = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if c & 127 == 127 else -x if c & 128 else x
    return out


def e4m3_round(x):
    """Codes of finite x, |x| <= 448, to nearest even; NaN of what is not finite."""
    x = np.asarray(x, dtype=np.float64)
    table = e4m3_values()[:127]
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.minimum(np.searchsorted(table, a), 126)
    lo = np.maximum(hi - 1, 0)
    low, high = a - table[lo], table[hi] - a
    code = np.where((low < high) | ((low == high) & (lo % 2 == 0)), lo, hi)
    code = np.where(a == table[hi], hi, code)
    return np.where(np.isfinite(x), code + 128 * np.signbit(x), 127).astype(np.uint8)


def scale_byte(top):
    """The smallest b >= 1 with top <= 448 * 2^(b - 127)."""
    b = 1
    while b < 254 and top > 448 * 2.0 ** (b - 127):
        b += 1
    return b


def append_q8(x, codes, scales, q_offsets, kv_lens, page_table):
    """Stores x [N, Hk, D] (normed and rotated) in codes [pages, Hk, page, D] and scales [pages, Hk, page / 16], uint8,
    in place, for good offsets, lengths and pages; a page outside the cache is passed over. Returns the exact values in
    code units (NaN where nothing was stored) and, in their shape, the largest |x| of each block and head."""
    pages, Hk, page, D = codes.shape
    exact, tops = np.full(codes.shape, np.nan), np.zeros(scales.shape)
    values = e4m3_values()
    for s, held in enumerate(kv_lens):
        m = q_offsets[s + 1] - q_offsets[s]
        start = max(held - m, 0)
        for first in range(start // 16 * 16, held if m else 0, 16):
            pg = int(page_table[s][first // page])
            if not 0 <= pg < pages:
                continue
            lo, hi, at = max(first, start), min(first + 16, held), first % page
            token = q_offsets[s + 1] - held + lo
            for h in range(Hk):
                new = x[token:token + hi - lo, h].astype(np.float64)
                fine = np.isfinite(new)
                top = np.abs(new[fine]).max(initial=0.0)
                b, had = scale_byte(top), int(scales[pg, h, at // 16])
                if lo > first:
                    b = max(b, had)
                    if b > had:
                        old = values[codes[pg, h, at:at + lo - first]]
                        sign = codes[pg, h, at:at + lo - first] & 128
                        codes[pg, h, at:at + lo - first] = e4m3_round(old * 2.0 ** (had - b)) | sign
                tops[pg, h, at // 16] = top
                scales[pg, h, at // 16] = b
                units = new / 2.0 ** (b - 127)
                exact[pg, h, at + lo - first:at + hi - first] = units
                codes[pg, h, at + lo - first:at + hi - first] = e4m3_round(units)
    return exact, tops
