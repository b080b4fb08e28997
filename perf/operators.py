"""Cases of the user-history attention operators: what is timed, on which inputs, and what the result is.

The operators serve a recommendation model that encodes a user's event history as a sequence: per-head norms of queries and
keys with the position rotation (and its backward pass, for training), appending keys and values to a paged cache, and the
attention of new tokens over that cache. `run` computes them in plain torch, or with `own` through the framework's entry points.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"
EPS = 1e-6


def listed():
    return [
        # a handful of fresh events of one request: latency
        dict(name="norm rope, few tokens", op="norm_rope", tokens=5, q_heads=8, kv_heads=2, dim=64, rot=64, axes=1,
             inter=False, norm=True, type="f16"),
        # a training batch of long histories, positions by index and time
        dict(name="norm rope, training batch", op="norm_rope", tokens=16384, q_heads=32, kv_heads=8, dim=128, rot=128,
             axes=2, inter=False, norm=True, type="bf16"),
        # the gradient in fp32, half of each head rotated, neighbouring pairs, an odd number of tokens
        dict(name="norm rope backward, fp32", op="norm_rope_bwd", tokens=4099, q_heads=12, kv_heads=4, dim=64, rot=32,
             axes=1, inter=True, norm=True, type="f32"),
        # the gradient of the training batch
        dict(name="norm rope backward, training", op="norm_rope_bwd", tokens=16384, q_heads=32, kv_heads=8, dim=128,
             rot=128, axes=2, inter=False, norm=True, type="bf16"),
        # one new event for each of 96 users
        dict(name="append, one token each", op="append", seqs=96, q_max=1, kv_max=4096, page=16, q_heads=16, kv_heads=4,
             dim=128, rot=128, axes=1, inter=False, norm=True, type="bf16", lens=1),
        # histories filled in chunks of up to 2048 events
        dict(name="append, chunks", op="append", seqs=12, q_max=2048, kv_max=8192, page=64, q_heads=32, kv_heads=8,
             dim=128, rot=64, axes=1, inter=True, norm=False, type="f16", lens=2),
        # one new event over a short history: latency
        dict(name="attention, one short", op="attention", seqs=1, q_max=1, kv_max=301, page=16, q_heads=8, kv_heads=2,
             dim=64, causal=True, window=0, type="f16", lens=3),
        # a serving batch: one new event each, histories from one event to 16k
        dict(name="attention, serving batch", op="attention", seqs=64, q_max=1, kv_max=16384, page=64, q_heads=32,
             kv_heads=8, dim=128, causal=True, window=0, type="bf16", lens=4),
        # one life-long history
        dict(name="attention, one long", op="attention", seqs=1, q_max=1, kv_max=131009, page=16, q_heads=16, kv_heads=2,
             dim=128, causal=True, window=0, type="bf16", lens=5),
        # ranking: up to 257 candidates per user, each over the user's whole history
        dict(name="attention, candidates", op="attention", seqs=24, q_max=257, kv_max=1500, page=32, q_heads=4,
             kv_heads=4, dim=64, causal=False, window=0, type="bf16", lens=6),
        # ragged chunks that see the last 1024 events, wide heads
        dict(name="attention, ragged window", op="attention", seqs=12, q_max=513, kv_max=6000, page=16, q_heads=8,
             kv_heads=4, dim=256, causal=True, window=1024, type="f16", lens=7),
        # long chunks over long histories
        dict(name="attention, long chunks", op="attention", seqs=4, q_max=2048, kv_max=8192, page=64, q_heads=32,
             kv_heads=8, dim=128, causal=True, window=0, type="bf16", lens=8),
    ]


def _between(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        for k in w:
            most[k] = max(most.get(k, 0), w[k])
    while True:
        op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "attention", "attention", "attention"])
        kv_heads, dim = rng.choice([1, 2, 3, 4, 8]), rng.choice([32, 64, 128, 256])
        c = dict(op=op, q_heads=kv_heads * rng.choice([1, 2, 3, 4, 8]), kv_heads=kv_heads, dim=dim)
        if op == "attention":
            c.update(type=rng.choice(["f16", "bf16"]), seqs=_between(rng, 1, 64), q_max=rng.choice([1, _between(rng, 1, 2048)]),
                     kv_max=_between(rng, 1, 131072), page=rng.choice([16, 32, 64, 128]), causal=rng.random() < 0.75)
            c["window"] = _between(rng, 1, 4096) if c["causal"] and rng.random() < 0.3 else 0
        else:
            c.update(rot=rng.choice([dim, dim, dim // 2]), axes=rng.choice([1, 1, 2, 3]), inter=rng.random() < 0.5,
                     norm=rng.random() < 0.75)
            if op == "append":
                c.update(type=rng.choice(["f16", "bf16"]), seqs=_between(rng, 1, 128), q_max=rng.choice([1, _between(rng, 1, 2048)]),
                         kv_max=_between(rng, 1, 16384), page=rng.choice([16, 32, 64, 128]))
            else:
                c.update(type=rng.choice(["f32", "f16", "bf16"]), tokens=_between(rng, 1, 16384))
        if "seqs" in c:
            c["q_max"] = min(c["q_max"], c["kv_max"])
            c["lens"] = rng.randrange(1 << 30)
            # scores of the padded batch, and the padded histories, that the plain form holds at once
            if c["seqs"] * c["q_heads"] * c["q_max"] * c["kv_max"] > 1 << 31 or c["seqs"] * c["kv_max"] * kv_heads * dim > 1 << 30:
                continue
        w = work(c)
        if all(w[k] <= most[k] for k in w):
            return c


def _lengths(c):
    """New tokens and history length (the new ones included) of each sequence: the first has both at their largest."""
    rng = random.Random(c["lens"])
    q, kv = [], []
    for s in range(c["seqs"]):
        n = c["q_max"] if s == 0 or c["q_max"] == 1 else rng.randint(1, c["q_max"])
        h = c["kv_max"] if s == 0 else _between(rng, max(1, c["kv_max"] // 32), c["kv_max"])
        q.append(n)
        kv.append(max(n, h))
    return q, kv


def _visible(c):
    """Pairs of a new token and a history entry that it sees, and history entries that any of a sequence's tokens sees."""
    pairs = entries = 0
    for n, h in zip(*_lengths(c)):
        if not c["causal"]:
            pairs, entries = pairs + n * h, entries + h
        elif c["window"]:
            pairs += sum(min(c["window"], p + 1) for p in range(h - n, h))
            entries += min(h, n - 1 + c["window"])
        else:
            pairs += n * h - n * (n - 1) // 2
            entries += h
    return pairs, entries


def work(case):
    c, size = case, 4 if case["type"] == "f32" else 2
    heads, d = c["q_heads"] + c["kv_heads"], c["dim"]
    if c["op"] == "attention":
        pairs, entries = _visible(c)
        n = sum(_lengths(c)[0])
        return {"bytes": 2 * n * c["q_heads"] * d * size + 4 * n * c["q_heads"] + 2 * entries * c["kv_heads"] * d * size,
                "flops": 4 * pairs * c["q_heads"] * d}
    if c["op"] == "append":
        n = sum(_lengths(c)[0])
        return {"bytes": 2 * n * (heads + c["kv_heads"]) * d * size, "flops": 10 * n * heads * d}
    n, norm = c["tokens"], c["norm"]
    if c["op"] == "norm_rope":
        return {"bytes": 2 * n * heads * d * size + 4 * n * c["axes"], "flops": 10 * n * heads * d}
    return {"bytes": (3 if norm else 2) * n * heads * d * size + 4 * n * c["axes"], "flops": 20 * n * heads * d}


def _sections(c):
    """How many of the rotation's frequencies each position axis turns."""
    pairs, a = c["rot"] // 2, c["axes"]
    return [pairs // a + (i < pairs % a) for i in range(a)]


def prepare(case, seed):
    c, t = case, TYPES[case["type"]]
    g = torch.Generator(DEV).manual_seed(seed)
    hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]

    def normal(*shape, dtype=t):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)

    s = {"case": c}
    if "seqs" in c:
        q_lens, kv_lens = _lengths(c)
        n, width = sum(q_lens), -(-max(kv_lens) // c["page"])
        counts = torch.tensor([-(-h // c["page"]) for h in kv_lens], device=DEV)
        used = int(sum(-(-h // c["page"]) for h in kv_lens))
        order = torch.randperm(used + 3, generator=g, device=DEV).to(torch.int32)
        column = torch.arange(width, device=DEV)
        entry = (counts.cumsum(0) - counts)[:, None] + column
        s["page_table"] = torch.where(column < counts[:, None], order[entry.clamp(max=used - 1)], torch.full_like(entry, -1, dtype=torch.int32))
        s["q_offsets"] = torch.tensor([0] + q_lens, device=DEV).cumsum(0).to(torch.int32)
        s["kv_lens"] = torch.tensor(kv_lens, device=DEV, dtype=torch.int32)
        s["max_q"], s["max_kv"] = max(q_lens), max(kv_lens)
        s["k_cache"] = normal(used + 3, hk, c["page"], d)
        s["v_cache"] = normal(used + 3, hk, c["page"], d)
    else:
        n = c["tokens"]
    qkv = normal(n, (hq + 2 * hk) * d)  # one projection's output, the heads next to each other
    s["q"] = qkv[:, : hq * d].view(n, hq, d)
    if c["op"] != "attention":
        s["k"] = qkv[:, hq * d : (hq + hk) * d].view(n, hk, d)
        s["v"] = qkv[:, (hq + hk) * d :].view(n, hk, d)
        s["sections"] = _sections(c)
        s["axis"] = torch.tensor([a for a, many in enumerate(s["sections"]) for _ in range(many)], device=DEV)
        s["inv_freq"] = (10000.0 ** (-torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64) * 2 / c["rot"])).float()
        # the index in the history, then the time and the like: whole numbers that reach far
        s["positions"] = torch.randint(0, 1 << 17, (c["axes"], n), generator=g, device=DEV, dtype=torch.int32)
        s["w_q"] = 1 + 0.1 * normal(d, dtype=torch.float32) if c["norm"] else None
        s["w_k"] = 1 + 0.1 * normal(d, dtype=torch.float32) if c["norm"] else None
    if c["op"] == "norm_rope_bwd":
        s["d_q_out"], s["d_k_out"] = normal(n, hq, d), normal(n, hk, d)
    return s


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def _own(s):
    from sparse_embedding_lookup_dlrm_amd import ops

    c = s["case"]
    if c["op"] == "attention":
        out, lse = ops.paged_attn(s["q"], s["k_cache"], s["v_cache"], s["q_offsets"], s["kv_lens"], s["page_table"],
                                  causal=c["causal"], window=c["window"], max_q=s["max_q"], max_kv=s["max_kv"], want_lse=True)
        return {"out": out, "lse": lse}
    how = dict(eps=EPS, sections=s["sections"], interleaved=c["inter"])
    if c["op"] == "norm_rope":
        q, k = ops.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["w_q"], s["w_k"], **how)
        return {"q": q, "k": k}
    if c["op"] == "append":
        q = ops.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["q_offsets"], s["kv_lens"], s["page_table"], q=s["q"],
                          positions=s["positions"], inv_freq=s["inv_freq"], w_q=s["w_q"], w_k=s["w_k"], **how)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    d_q, d_k, d_w_q, d_w_k = ops.qk_norm_rope_bwd(s["d_q_out"], s["d_k_out"], s["q"], s["k"], s["positions"], s["inv_freq"],
                                                  s["w_q"], s["w_k"], **how)
    return {"d_q": d_q, "d_k": d_k, "d_w_q": d_w_q, "d_w_k": d_w_k}


# The plain forms.


def _angles(s):
    """cos and sin of each token's angles [N, 1, R/2], the angles in 64 bits: positions reach far."""
    a = s["positions"][s["axis"]].T.double() * s["inv_freq"].double()
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _rotate(x, cos, sin, inter):
    r = 2 * cos.shape[-1]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if inter else (x[..., : r // 2], x[..., r // 2 : r])
    y = [a * cos - b * sin, a * sin + b * cos]
    y = torch.stack(y, -1).flatten(-2) if inter else torch.cat(y, -1)
    return torch.cat([y, x[..., r:]], -1)


def _norm_rope_one(x, w, cos, sin, inter):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w
    return _rotate(y, cos, sin, inter).to(x.dtype)


def _norm_rope(s):
    cos, sin = _angles(s)
    inter = s["case"]["inter"]
    return {"q": _norm_rope_one(s["q"], s["w_q"], cos, sin, inter), "k": _norm_rope_one(s["k"], s["w_k"], cos, sin, inter)}


def _norm_rope_bwd_one(dy, x, w, cos, sin, inter):
    g = _rotate(dy.float(), cos, -sin, inter)
    if w is None:
        return g.to(x.dtype), None
    x32 = x.float()
    r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
    xn, gw = x32 * r, g * w
    dx = r * (gw - xn * (gw * xn).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * xn).sum((0, 1))


def _norm_rope_bwd(s):
    cos, sin = _angles(s)
    inter = s["case"]["inter"]
    d_q, d_w_q = _norm_rope_bwd_one(s["d_q_out"], s["q"], s["w_q"], cos, sin, inter)
    d_k, d_w_k = _norm_rope_bwd_one(s["d_k_out"], s["k"], s["w_k"], cos, sin, inter)
    return {"d_q": d_q, "d_k": d_k, "d_w_q": d_w_q, "d_w_k": d_w_k}


def _tokens(s):
    """Each new token's sequence and its place in it."""
    n = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(s["q_offsets"][1:], n, right=True)
    return seq, n - s["q_offsets"][seq]


def _append(s):
    both = _norm_rope(s)
    seq, i = _tokens(s)
    at = (s["kv_lens"] - s["q_offsets"].diff())[seq] + i
    page = s["case"]["page"]
    pages = s["page_table"][seq, at // page].long()
    s["k_cache"][pages, :, at % page] = both["k"]
    s["v_cache"][pages, :, at % page] = s["v"]
    return {"q": both["q"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attention(s):
    c = s["case"]
    hk, d, group = c["kv_heads"], c["dim"], c["q_heads"] // c["kv_heads"]
    pages = s["page_table"].clamp(min=0).long()
    k, v = (s[x][pages].permute(0, 2, 1, 3, 4).flatten(2, 3).float() for x in ("k_cache", "v_cache"))  # [S, Hk, keys, D]
    seq, i = _tokens(s)
    q = torch.zeros(c["seqs"], s["max_q"], c["q_heads"], d, device=DEV)
    q[seq, i] = s["q"].float()
    q = q.unflatten(2, (hk, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [S, Hk, tokens * group, D]
    scores = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(d**-0.5).unflatten(2, (s["max_q"], group))
    lens = s["kv_lens"][:, None, None]
    at = (lens - s["q_offsets"].diff()[:, None, None]) + torch.arange(s["max_q"], device=DEV)[None, :, None]
    key = torch.arange(k.shape[2], device=DEV)
    hidden = key >= lens
    if c["causal"]:
        hidden = hidden | (key > at)
    if c["window"]:
        hidden = hidden | (key <= at - c["window"])
    scores.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), v).unflatten(2, (s["max_q"], group)) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log())[..., 0]
    # [S, Hk, tokens, group, ..] -> [N, Hq, ..]
    out, lse = (x.permute(0, 2, 1, 3, *range(4, x.dim())).flatten(2, 3)[seq, i] for x in (out, lse))
    return {"out": out.to(s["q"].dtype), "lse": lse}


_PLAIN = {"norm_rope": _norm_rope, "norm_rope_bwd": _norm_rope_bwd, "append": _append, "attention": _attention}


# The definitions in 64 bits, written apart from the plain forms.


def _turns(c, s, back=False):
    """One complex factor for each token and frequency."""
    first, parts = 0, []
    for a, many in enumerate(s["sections"]):
        w = s["inv_freq"][first : first + many].double()
        parts.append(torch.outer(s["positions"][a].double(), w))
        first += many
    angle = torch.cat(parts, 1)
    return torch.polar(torch.ones_like(angle), -angle if back else angle).unsqueeze(1)


def _turned(c, x, factor):
    half = c["rot"] // 2
    head = x[..., : c["rot"]]
    pairs = head.unflatten(-1, (half, 2)) if c["inter"] else head.unflatten(-1, (2, half)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * factor)
    y = x.clone()
    y[..., : c["rot"]] = z.flatten(-2) if c["inter"] else z.transpose(-1, -2).flatten(-2)
    return y


def _exact_norm(x, w):
    x = x.double()
    if w is None:
        return x, None, None
    size = torch.sqrt(torch.sum(x**2, -1, keepdim=True) / x.shape[-1] + EPS)
    return x / size * w.double(), x / size, size


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm_rope":
        f = _turns(c, s)
        return {x: _turned(c, _exact_norm(s[x], s["w_" + x])[0], f) for x in ("q", "k")}
    if c["op"] == "norm_rope_bwd":
        f, found = _turns(c, s, back=True), {}
        for x in ("q", "k"):
            g = _turned(c, s["d_%s_out" % x].double(), f)
            w, (_, unit, size) = s["w_" + x], _exact_norm(s[x], s["w_" + x])
            found["d_w_" + x] = None
            if w is not None:
                found["d_w_" + x] = torch.einsum("nhd,nhd->d", g, unit)
                g = g * w.double()
                g = (g - unit * torch.sum(g * unit, -1, keepdim=True) / c["dim"]) / size
            found["d_" + x] = g
        return found
    q_lens, kv_lens = _lengths(c)
    page = c["page"]
    if c["op"] == "append":
        f = _turns(c, s)
        k = _turned(c, _exact_norm(s["k"], s["w_k"])[0], f)
        caches = {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
        first = 0
        for b, (n, h) in enumerate(zip(q_lens, kv_lens)):
            at = torch.arange(h - n, h, device=DEV)
            pages = s["page_table"][b].long()[torch.div(at, page, rounding_mode="floor")]
            caches["k_cache"][pages, :, at % page] = k[first : first + n]
            caches["v_cache"][pages, :, at % page] = s["v"][first : first + n].double()
            first += n
        return {"q": _turned(c, _exact_norm(s["q"], s["w_q"])[0], f), **caches}
    outs, sums, first = [], [], 0
    group = c["q_heads"] // c["kv_heads"]
    for b, (n, h) in enumerate(zip(q_lens, kv_lens)):
        pages = s["page_table"][b, : -(-h // page)].long()
        k, v = (s[x][pages].double().transpose(1, 2).reshape(-1, c["kv_heads"], c["dim"])[:h] for x in ("k_cache", "v_cache"))
        q = s["q"][first : first + n].double()
        first += n
        row, col = torch.arange(h - n, h, device=DEV)[:, None], torch.arange(h, device=DEV)[None]
        seen = (col <= row) & (col > row - (c["window"] or h + 1)) if c["causal"] else torch.ones(n, h, dtype=torch.bool, device=DEV)
        o, l = [], []
        for head in range(c["q_heads"]):
            z = (q[:, head] @ k[:, head // group].T.contiguous()) / math.sqrt(c["dim"])
            z = torch.where(seen, z, torch.full_like(z, -math.inf))
            l.append(torch.logsumexp(z, 1))
            o.append(torch.softmax(z, 1) @ v[:, head // group].contiguous())
        outs.append(torch.stack(o, 1))
        sums.append(torch.stack(l, 1))
    return {"out": torch.cat(outs), "lse": torch.cat(sums)}
