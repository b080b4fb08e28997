"""Encoding users' event histories as sequences beside the embedding bags.

    python examples/user_history.py

A user's events are item ids. Their table rows are projected to queries, keys and values; the keys (normed
and rotated by place and time) and the values go to a paged cache, so that a new event costs one append
and one attention over the user's history, not the history again. The last event's attention output is the
user's vector, a feature of the pairwise interaction like a pooled bag. Candidates are ranked by letting each
attend to the whole history without being stored. Training the per-head norms takes the backward of norm and
rotation.
"""
from __future__ import annotations

import os
import sys
from typing import List, Sequence

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from sparse_embedding_lookup_dlrm_amd import ops  # noqa: E402


class HistoryCache:
    """Paged keys and values of many users on one GPU: hands out pages as histories grow."""

    def __init__(self, users: int, pages: int, kv_heads: int, page: int, dim: int, max_events: int, dtype, device):
        self.page = page
        self.k = torch.zeros((pages, kv_heads, page, dim), dtype=dtype, device=device)
        self.v = torch.zeros_like(self.k)
        self.free = list(range(pages))
        self.held = [0] * users
        self.pages: List[List[int]] = [[] for _ in range(users)]
        self.width = -(-max_events // page)

    def grow(self, users: Sequence[int], new: Sequence[int]):
        """Room for new[i] events of users[i]; returns q_offsets, kv_lens and page table of the call and its
        largest numbers of new and of held events. Without room nothing changes."""
        if len(set(users)) != len(users):
            raise ValueError("a user's new events go in one sequence")
        for u, n in zip(users, new):
            if self.held[u] + n > self.width * self.page:
                raise ValueError(f"user {u} would hold {self.held[u] + n} events, there is room for {self.width * self.page}")
        pages = sum(-(-(self.held[u] + n) // self.page) - len(self.pages[u]) for u, n in zip(users, new))
        if pages > len(self.free):
            raise ValueError(f"{pages} more pages are needed, {len(self.free)} are free")
        for u, n in zip(users, new):
            self.held[u] += n
            while len(self.pages[u]) * self.page < self.held[u]:
                self.pages[u].append(self.free.pop())
        return self.batch(users, new)

    def batch(self, users: Sequence[int], rows: Sequence[int]):
        dev = self.k.device
        table = torch.full((len(users), self.width), -1, dtype=torch.int32)
        for i, u in enumerate(users):
            table[i, :len(self.pages[u])] = torch.tensor(self.pages[u], dtype=torch.int32)
        offsets = torch.tensor([0] + list(rows)).cumsum(0).to(torch.int32)
        lens = torch.tensor([self.held[u] for u in users], dtype=torch.int32)
        most = dict(max_q=max(rows), max_kv=max(self.held[u] for u in users))
        return (offsets.to(dev), lens.to(dev), table.to(dev)), most


class HistoryEncoder:
    """One attention layer over item embeddings: a joint projection, per-head norms, and a rotation whose first
    pairs turn by the event's place in the history and whose last ones by its hour."""

    def __init__(self, items: int, width: int, q_heads: int, kv_heads: int, dim: int, dtype=torch.bfloat16,
                 device="cuda", seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        self.q_heads, self.kv_heads, self.dim = q_heads, kv_heads, dim
        self.items = torch.randn((items, width), generator=g).to(device, dtype)
        proj = torch.randn((width, (q_heads + 2 * kv_heads) * dim), generator=g) * width ** -0.5
        self.proj = proj.to(device, dtype)
        self.w_q = torch.ones(dim, device=device)
        self.w_k = torch.ones(dim, device=device)
        pairs = dim // 2
        self.sections = [pairs - pairs // 4, pairs // 4]
        self.inv_freq = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().to(device)

    def project(self, ids: torch.Tensor):
        """q, k and v of item ids: slices of one product, not copied."""
        x = self.items[ids.long()] @ self.proj
        n, a, b = x.shape[0], self.q_heads * self.dim, (self.q_heads + self.kv_heads) * self.dim
        return (x[:, :a].view(n, -1, self.dim), x[:, a:b].view(n, -1, self.dim), x[:, b:].view(n, -1, self.dim))

    def turn(self, positions):
        return dict(positions=positions, inv_freq=self.inv_freq, w_q=self.w_q, w_k=self.w_k, sections=self.sections)

    def step(self, cache: HistoryCache, users, ids, hours, new):
        """Appends new[i] events of each user and returns the attention outputs of all of them
        [events, q_heads * dim]. ids and hours hold the users' events one after the other."""
        before = [cache.held[u] for u in users]
        (offsets, lens, table), most = cache.grow(users, new)
        place = torch.cat([torch.arange(b, b + n) for b, n in zip(before, new)]).to(ids.device, torch.int32)
        q, k, v = self.project(ids)
        q = ops.kv_append(k, v, cache.k, cache.v, offsets, lens, table, q=q,
                          **self.turn(torch.stack([place, hours.to(torch.int32)])))
        return ops.paged_attn(q, cache.k, cache.v, offsets, lens, table, **most).flatten(1)

    def rank(self, cache: HistoryCache, users, ids, hours, many):
        """Candidates (many[i] for each user) over the whole histories; nothing is stored. A candidate takes the
        place after the last event."""
        (offsets, lens, table), most = cache.batch(users, many)
        place = torch.cat([torch.full((n,), cache.held[u]) for u, n in zip(users, many)]).to(ids.device, torch.int32)
        q, k, _ = self.project(ids)
        q, _ = ops.qk_norm_rope(q, k, torch.stack([place, hours.to(torch.int32)]), self.inv_freq, self.w_q, self.w_k,
                                sections=self.sections)
        return ops.paged_attn(q, cache.k, cache.v, offsets, lens, table, causal=False, **most).flatten(1)

    def train_norms(self, ids, place, hours, d_q, d_k, lr: float):
        """One SGD step on the norm weights from the gradients of the normed and rotated queries and keys;
        returns the gradients of the projection's q and k."""
        q, k, _ = self.project(ids)
        pos = torch.stack([place.to(torch.int32), hours.to(torch.int32)])
        g_q, g_k, g_w_q, g_w_k = ops.qk_norm_rope_bwd(d_q, d_k, q, k, pos, self.inv_freq, self.w_q, self.w_k,
                                                      sections=self.sections)
        self.w_q -= lr * g_w_q
        self.w_k -= lr * g_w_k
        return g_q, g_k


def main() -> None:
    dev = "cuda"
    enc = HistoryEncoder(items=10_000, width=128, q_heads=8, kv_heads=2, dim=64)
    users = 6
    cache = HistoryCache(users, pages=256, kv_heads=2, page=16, dim=64, max_events=512, dtype=torch.bfloat16,
                         device=dev)
    g = torch.Generator().manual_seed(1)
    past = [200, 3, 77, 120, 1, 64]
    ids = torch.randint(0, 10_000, (sum(past),), generator=g, dtype=torch.int32).to(dev)
    hours = torch.cat([torch.arange(n) * 7 for n in past]).to(dev)
    enc.step(cache, range(users), ids, hours, past)  # the histories so far, one ragged chunk

    # one new event of every user: its output is the user's vector
    ids = torch.randint(0, 10_000, (users,), generator=g, dtype=torch.int32).to(dev)
    now = torch.tensor([n * 7 for n in past], device=dev)
    user = enc.step(cache, range(users), ids, now, [1] * users).float()
    print("user vectors", tuple(user.shape))

    # the vectors join the pairwise interaction like pooled bags, a head pair to a feature
    e0 = torch.randn((users, 128), generator=g).to(dev)
    out = ops.interact(e0, user.view(users, -1, 128).contiguous())
    print("interaction", tuple(out.shape))

    # candidates
    many = [5, 0, 12, 3, 7, 1]
    ids = torch.randint(0, 10_000, (sum(many),), generator=g, dtype=torch.int32).to(dev)
    hours = torch.cat([torch.full((n,), past[u] * 7 + 1) for u, n in enumerate(many)]).to(dev)
    cand = enc.rank(cache, range(users), ids, hours, many)
    owner = torch.repeat_interleave(torch.arange(users), torch.tensor(many)).to(dev)
    score = (cand.float() * user[owner]).sum(1)
    print("best candidates", [int(score[owner == u].argmax()) if n else None for u, n in enumerate(many)])

    # a step on the norm weights
    n = 64
    ids = torch.randint(0, 10_000, (n,), generator=g, dtype=torch.int32).to(dev)
    d_q = torch.randn((n, 8, 64), generator=g).to(dev, torch.bfloat16)
    d_k = torch.randn((n, 2, 64), generator=g).to(dev, torch.bfloat16)
    g_q, _ = enc.train_norms(ids, torch.arange(n, device=dev), torch.arange(n, device=dev) * 7, d_q, d_k, 1e-3)
    print("norm weights moved by", float((enc.w_q - 1).abs().max()), "query gradients", tuple(g_q.shape))


if __name__ == "__main__":
    main()
