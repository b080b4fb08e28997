"""Bad offsets of sequences in the user-history operators: which tokens the append stores, and that the
attention takes the same sequences. Caches without pages, and strides that are never taken."""
import pytest
import torch

from gpu_util import need_gpu
from history_util import rand
from sparse_embedding_lookup_dlrm_amd import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def sequences_of(offsets, n):
    """The contract: sequence s has its tokens if its offsets ascend and stay in [0, n] and between the first
    and the last offset. Returns {sequence: (first, last)}, the empty ones left out."""
    lo, hi = max(0, offsets[0]), min(n, offsets[-1])
    return {s: (a, b) for s, (a, b) in enumerate(zip(offsets, offsets[1:])) if lo <= a < b <= hi}


def many(seed):
    """1000 sequences of 0 to 3 tokens, some offsets replaced by ones far off or a few tokens off."""
    g = torch.Generator().manual_seed(seed)
    off = [0] + torch.randint(0, 4, (1000,), generator=g).cumsum(0).tolist()
    n = off[-1]
    for i in torch.randint(1, 1000, (12,), generator=g).tolist():
        off[i] = [10 ** 6, -5, off[i] + 4, max(0, off[i] - 4)][int(torch.randint(0, 4, (1,), generator=g))]
    return off, n


OFFSETS = [([0, 50, 3, 6], 6), ([0, 2, -7, 4, 6], 6), ([0, 3, 2, 6], 6), ([5, 2, 8], 8), ([0, 50, 3], 60),
           ([0, 2, 100], 6), ([-3, 2, 6], 6), ([0, 4, 4, 1, 6], 6), many(1), many(2), many(3)]


@pytest.mark.parametrize("case", range(len(OFFSETS)))
def test_append_and_attention_take_the_same_sequences(case):
    """Every token of an accepted sequence is stored in its slot (in overlapping sequences, in one of them) and
    nothing else; the attention's results are those of a call with each accepted sequence alone."""
    offsets, n = OFFSETS[case]
    S, Hk, D, page = len(offsets) - 1, 2, 64, 16
    good = sequences_of(offsets, n)
    longest = max([b - a for a, b in good.values()] + [1])
    lens = [longest + 9 + s % 5 for s in range(S)]
    width = -(-max(lens) // page)
    table = torch.randperm(S * width, generator=torch.Generator().manual_seed(case)).to(torch.int32).view(S, width)
    k, v, q = (rand((n, h, D), "bf16", 10 * case + i) for i, h in enumerate((Hk, Hk, 4)))
    kc0, vc0 = (rand((S * width, Hk, page, D), "bf16", 10 * case + 5 + i) for i in range(2))
    kc, vc, status = kc0.cuda(), vc0.cuda(), i32([0])
    ops.kv_append(k.cuda(), v.cuda(), kc, vc, i32(offsets), i32(lens), table.cuda(), status=status)
    assert status.item() == ops.STATUS_BAD_OFFSETS
    kc_host, vc_host = kc.cpu(), vc.cpu()
    slots = {t: [] for t in range(n)}
    for s, (a, b) in good.items():
        for t in range(a, b):
            at = lens[s] - b + t
            slots[t].append((int(table[s, at // page]), slice(None), at % page))
    for t, found in slots.items():
        if len(found) == 1:
            kc0[found[0]], vc0[found[0]] = k[t], v[t]
        elif found:
            assert sum(torch.equal(kc_host[at], k[t]) and torch.equal(vc_host[at], v[t]) for at in found) == 1
            for at in found:
                kc0[at], vc0[at] = kc_host[at], vc_host[at]
    assert torch.equal(kc_host.view(torch.int16), kc0.view(torch.int16))
    assert torch.equal(vc_host.view(torch.int16), vc0.view(torch.int16))

    status.zero_()
    out = torch.full((n, 4, D), 3.0, dtype=torch.bfloat16, device="cuda")
    how = dict(max_q=longest, max_kv=1)  # one part to a history: a row's sums do not depend on the other sequences
    ops.paged_attn(q.cuda(), kc, vc, i32(offsets), i32(lens), table.cuda(), out=out, status=status, **how)
    assert status.item() == ops.STATUS_BAD_OFFSETS
    want = torch.full_like(out, 3.0)
    for s, (a, b) in good.items():
        want[a:b] = ops.paged_attn(q[a:b].cuda(), kc, vc, i32([0, b - a]), i32(lens[s:s + 1]), table[s:s + 1].cuda(), **how)
    once = torch.tensor([len(slots[t]) <= 1 for t in range(n)], device="cuda")
    assert torch.equal(out[once], want[once])


@pytest.mark.parametrize("max_q", [1, 40])
def test_attention_over_a_cache_without_pages(max_q):
    """Bad offsets and lengths are reported as with pages, bad pages only where a token would see an entry; the
    tokens see nothing."""
    S, B, P = 2, ops.STATUS_BAD_OFFSETS, ops.STATUS_BAD_PAGE
    q = rand((6, 4, 64), "bf16", 1).cuda()
    table = torch.full((S, 3), -1, dtype=torch.int32, device="cuda")
    for offsets, lens, want in (([0, 2, 6], [9, 8], P), ([0, 2, 6], [0, 0], 0), ([0, 0, 0], [9, 8], 0),
                                ([0, 6, 6], [0, 8], 0), ([0, 9, 6], [5, 5], B), ([0, 2, 6], [0, -1], B),
                                ([0, 2, 6], [0, 10 ** 6], B | P), ([0, 2, 6], [1, -3], B | P)):
        for pages in (0, 1):  # no page at all, and one that no table names
            cache = torch.zeros((pages, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
            status = i32([0])
            out, lse = torch.full_like(q, 3.0), torch.full((6, 4), 3.0, device="cuda")
            ops.paged_attn(q, cache, cache, i32(offsets), i32(lens), table, out=out, lse=lse, want_lse=True,
                           status=status, max_q=max_q)
            assert status.item() == want, (offsets, lens, pages)
            taken = torch.zeros(6, dtype=torch.bool)
            for a, b in sequences_of(offsets, 6).values():
                taken[a:b] = True
            assert (out[taken.cuda()] == 0).all() and (lse[taken.cuda()] == -float("inf")).all()
            assert (out[~taken.cuda()] == 3).all() and (lse[~taken.cuda()] == 3).all()


def test_strides_of_single_pages_and_heads_are_not_looked_at():
    """One head, or one page, with any stride over it, another one in each cache."""
    q, k, v = (rand((3, h, 64), "bf16", i).cuda() for i, h in enumerate((2, 1, 1)))
    for pages, odd_k, odd_v in ((4, (1024, 7, 64, 1), (1024, 13, 64, 1)), (1, (3, 1024, 64, 1), (1024, 5, 64, 1))):
        kc, vc, want_k, want_v = (torch.zeros((pages, 1, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(4))
        args = i32([0, 3]), i32([9]), i32([[pages - 1]])
        ops.kv_append(k, v, want_k, want_v, *args)
        ops.kv_append(k, v, kc.as_strided(kc.shape, odd_k), vc.as_strided(vc.shape, odd_v), *args)
        assert torch.equal(kc, want_k) and torch.equal(vc, want_v) and kc.any()
        out = ops.paged_attn(q, kc.as_strided(kc.shape, odd_k), vc.as_strided(vc.shape, odd_v), *args)
        assert torch.equal(out, ops.paged_attn(q, want_k, want_v, *args))
