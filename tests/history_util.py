"""Inputs and tolerances of the user-history attention tests.

Tolerances count roundings: u = 2^-24 for a step in fp32, half(t) = eps / 2 for the rounding to a
type, relative to the magnitudes that the oracle returns, plus half of a subnormal step of fp16.
Norm and rotation: at most 16 products in a row and 5 joins in the sum of squares, halved by the
root (11 u), the root and two products (4 u), sine and cosine (4 u), the angle rounded to 2^-25 of a
half-turn (2 u), the rotation (3 u): 32 u covers them.
Attention: a score is off by (D + 8) u of sum |q||k| and by 8 u of its own size in the exponent; a
weight by that and by its rounding to the type; sums over n entries by (n + 32) u.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}


def half(t):
    return torch.finfo(TYPES[t]).eps / 2


def np64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, tol, what):
    got = np64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off; first at {i}: got {got[i]!r} ref {ref[i]!r} "
                             f"tolerance {np.broadcast_to(tol, ref.shape)[i]!r}")


def norm_rope_tol(t, ref, mag):
    return half(t) * np.abs(ref) + 32 * U * mag + TINY[t]


def attention_tol(t, ref, mag, size, count, D, v_max):
    """Tolerances of out and lse."""
    out, lse = ref
    n = count.astype(np.float64)
    top = np.where(np.isfinite(lse), np.abs(lse), 0.0) + np.log(np.maximum(n, 1))  # bounds |scale * m|
    weight = ((D + 8) * size + 8 * top) * U
    # fp16 weights are subnormal below 2^-22 of the largest: half a step is 2^-33 of it
    sub = n * 2.0 ** -33 * v_max if t == "f16" else 0 * n
    o = half(t) * (np.abs(out) + mag * (1 + half(t))) + (2 * weight + (n + 32) * U)[..., None] * mag + TINY[t] + sub[..., None]
    return o, weight + (n + 32) * U + 4 * U * top


def rand(shape, t, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(TYPES[t])


def sections_of(pairs, axes):
    return [pairs // axes + (i < pairs % axes) for i in range(axes)]


class Rope:
    """Positions, frequencies and weights of a norm and rotation, on the CPU."""

    def __init__(self, N, D, rot, axes, norm, seed, far=1 << 17):
        g = torch.Generator().manual_seed(seed + 77)
        self.positions = torch.randint(0, far, (axes, N), generator=g, dtype=torch.int32)
        self.inv_freq = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(rot, 1))).float() if rot else None
        self.sections = sections_of(rot // 2, axes)
        self.w_q = 1 + 0.2 * torch.randn(D, generator=g) if norm else None
        self.w_k = 1 + 0.2 * torch.randn(D, generator=g) if norm else None

    def angles(self):
        from oracle import history_oracle as ho

        freq = np.zeros(0) if self.inv_freq is None else self.inv_freq.numpy()
        return ho.angles(self.positions.numpy(), freq, self.sections)

    def dev(self):
        f = lambda x: None if x is None else x.cuda()
        return f(self.positions), f(self.inv_freq), f(self.w_q), f(self.w_k)


class History:
    """Sequences over a paged cache, on the CPU. Unused pages, and slots past each history, hold NaN."""

    def __init__(self, q_lens, kv_lens, Hq, Hk, D, page, t, seed, spare=3, fill=None, q_scale=1.0):
        self.q_lens, self.kv_lens, self.t = list(q_lens), list(kv_lens), t
        N = sum(q_lens)
        self.q = rand((N, Hq, D), t, seed, q_scale)
        self.q_offsets = torch.tensor([0] + self.q_lens).cumsum(0).to(torch.int32)
        counts = [-(-h // page) for h in kv_lens]
        width = max(counts + [1]) + 1
        total = sum(counts) + spare
        g = torch.Generator().manual_seed(seed + 1)
        order = torch.randperm(total, generator=g)
        self.page_table = torch.full((len(kv_lens), width), -1, dtype=torch.int32)
        self.k_cache = torch.full((total, Hk, page, D), float("nan"), dtype=TYPES[t])
        self.v_cache = torch.full((total, Hk, page, D), float("nan"), dtype=TYPES[t])
        kn, vn = rand((total, Hk, page, D), t, seed + 2), rand((total, Hk, page, D), t, seed + 3)
        at = 0
        for s, h in enumerate(kv_lens):
            for i in range(counts[s]):
                pg = int(order[at])
                at += 1
                self.page_table[s, i] = pg
                used = min(page, h - i * page)
                self.k_cache[pg, :, :used] = kn[pg, :, :used]
                self.v_cache[pg, :, :used] = vn[pg, :, :used]
        if fill is not None:
            self.k_cache = torch.nan_to_num(self.k_cache, nan=fill)
            self.v_cache = torch.nan_to_num(self.v_cache, nan=fill)

    def oracle(self, causal, window, scale):
        from oracle import history_oracle as ho

        return ho.attention(np64(self.q), np64(self.k_cache), np64(self.v_cache), self.q_offsets.tolist(),
                            self.kv_lens, self.page_table.tolist(), causal, window, scale)

    def args(self):
        return (self.q.cuda(), self.k_cache.cuda(), self.v_cache.cuda(), self.q_offsets.cuda(),
                torch.tensor(self.kv_lens, dtype=torch.int32).cuda(), self.page_table.cuda())


class History8(History):
    """Sequences over an 8-bit cache: codes and scale bytes, and in k_cache and v_cache the values they stand for. Slots
    past each history hold the code NaN, blocks without entries the byte 255 as well."""

    def __init__(self, *args, bytes_from=(118, 123), **kw):
        super().__init__(*args, **kw)
        g = torch.Generator().manual_seed(args[7] if len(args) > 7 else kw["seed"])
        pages, Hk, page, D = self.k_cache.shape
        self.scales = torch.randint(*bytes_from, (pages, Hk, page // 16, 2), generator=g, dtype=torch.int32).to(torch.uint8)
        self.codes = []
        for j, x in enumerate((self.k_cache, self.v_cache)):
            x = x.float().unflatten(2, (-1, 16))
            power = torch.exp2(self.scales[..., j].float() - 127)[..., None, None]
            code = (x / power).clamp(-448, 448).to(torch.float8_e4m3fn)
            self.codes.append(code.flatten(2, 3))
            empty = x.isnan().all(-1).all(-1)
            self.scales[..., j][empty] = 255
        self.values()

    def values(self):
        """k_cache and v_cache from the codes and scales."""
        power = self.scales.view(torch.float8_e8m0fnu).double().repeat_interleave(16, 2)
        self.k_cache, self.v_cache = (c.double() * power[..., j, None] for j, c in enumerate(self.codes))

    def args(self):
        return (self.q.cuda(), *(c.cuda() for c in self.codes), self.scales.view(torch.float8_e8m0fnu).cuda(),
                self.q_offsets.cuda(), torch.tensor(self.kv_lens, dtype=torch.int32).cuda(), self.page_table.cuda())
