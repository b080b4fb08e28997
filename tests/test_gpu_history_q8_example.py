"""The 8-bit operators together, as the example uses them: pages, append and attention without the host between them."""
import numpy as np
import pytest
import torch

from oracle import history_oracle as ho
from test_gpu_history_example import example  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def dense(cache, user, n):
    """Keys and values of a user's first n events [n, Hk, D], and where they are."""
    e = torch.arange(n, device="cuda")
    pages = cache.tables[user].long()[e // cache.page]
    power = torch.exp2(cache.scales.double() - 127).repeat_interleave(16, 2)
    return [(x.double() * power[..., j, None])[pages, :, e % cache.page] for j, x in enumerate((cache.k, cache.v))]


def test_steps_match_the_16_bit_cache(example):  # noqa: F811
    """The same events over both caches: keys and values differ by the rounding to 8 bits, half a step of which is 2^-4
    of the value or 2^-10 of the scale, and the scale is at most the block's largest value / 224."""
    enc = example.HistoryEncoder(items=500, width=64, q_heads=6, kv_heads=2, dim=64)
    past = [37, 1, 0, 20]
    whole = example.HistoryCache(4, pages=24, kv_heads=2, page=16, dim=64, max_events=64, dtype=torch.bfloat16, device="cuda")
    small = example.HistoryCache8(4, pages=24, kv_heads=2, page=16, dim=64, max_events=64, device="cuda")
    total = [0] * 4
    for step, new in enumerate((past, [1, 1, 1, 1], [2, 14, 0, 3])):
        users = [u for u in range(4) if new[u]]
        n = [new[u] for u in users]
        ids = torch.randint(0, 500, (sum(n),), dtype=torch.int32, generator=torch.Generator().manual_seed(step)).cuda()
        hours = torch.arange(sum(n), device="cuda") * 3 + step
        enc.step(whole, users, ids, hours, n)
        out = enc.step8(small, i32(users), ids, hours, i32(n), max(n))
        total = [a + b for a, b in zip(total, new)]
        assert small.held.tolist() == total == whole.held and small.status.item() == 0
        assert torch.isfinite(out).all()
        for u in users:
            at = torch.arange(total[u])
            pages = torch.tensor(whole.pages[u])[at // 16].cuda()
            for name, got in zip("kv", dense(small, u, total[u])):
                ref = getattr(whole, name)[pages, :, (at % 16).cuda()].double()
                top = ref.abs().amax() / 224
                # rounded again where a block's scale grew; and the 16-bit cache's own rounding
                assert ((got - ref).abs() <= 3 * (ref.abs() * 2.0 ** -4 + top * 2.0 ** -10) + ref.abs() * 2.0 ** -8).all()
        # the hours by slot
        last = len(hours) - 1
        u, place = users[-1], total[users[-1]] - 1
        slot = small.tables[u, place // 16].long() * 16 + place % 16
        assert small.hours[slot] == hours[last]
    # the attention over what the cache holds
    k, v = (torch.stack([F.pad(x, (0, 0, 0, 0, 0, 64 - len(x))) for x in xs]) for xs, F in
            ((d, torch.nn.functional) for d in zip(*(dense(small, u, total[u]) for u in range(4)))))
    q = torch.randn((4, 6, 64), device="cuda").to(torch.bfloat16)
    call, _, _ = small.grow(i32([0, 1, 2, 3]), i32([0, 0, 0, 0]), 0)
    offsets = i32([0, 1, 2, 3, 4])
    got = example.ops.paged_attn_q8(q, *small.parts(), offsets, *call[1:], causal=False)
    want, _, mag, _, _ = ho.attention(q.double().cpu().numpy(), k.cpu().numpy().transpose(0, 2, 1, 3), v.cpu().numpy().transpose(0, 2, 1, 3),
                                      offsets.tolist(), total, [[u] for u in range(4)], False, 0, 64 ** -0.5)
    # two roundings to bf16 (weights, result) and a hundredth for the sums
    assert (np.abs(got.double().cpu().numpy() - want) <= 2.0 ** -8 * (np.abs(want) + 1.01 * mag)).all()


def test_without_room_nothing_is_stored(example):  # noqa: F811
    enc = example.HistoryEncoder(items=500, width=64, q_heads=4, kv_heads=2, dim=64)
    cache = example.HistoryCache8(3, pages=4, kv_heads=2, page=16, dim=64, max_events=64, device="cuda")
    ids = torch.arange(40, dtype=torch.int32, device="cuda")
    enc.step8(cache, i32([0, 1]), ids[:30], ids[:30], i32([20, 10]), 20)
    before = [x.view(torch.uint8).clone() for x in (*cache.parts(), cache.hours, cache.held, cache.free, cache.count)]
    enc.step8(cache, i32([2, 1]), ids, ids, i32([33, 7]), 33)
    assert cache.status.item() == example.ops.STATUS_NO_ROOM
    for a, b in zip(before, (*cache.parts(), cache.hours, cache.held, cache.free, cache.count)):
        assert torch.equal(a, b.view(torch.uint8))
    cache.status.zero_()
    cache.drop(i32([0]), keep=i32([16]))
    enc.step8(cache, i32([2, 1]), ids[:30], ids[:30], i32([17, 6]), 17)
    assert cache.status.item() == 0 and cache.held.tolist() == [16, 16, 17] and cache.count.item() == 0


def test_tokens_without_a_slot_change_no_hours(example):  # noqa: F811
    """A padded batch whose one event takes slot 0, the place that tokens without a slot could be sent to."""
    enc = example.HistoryEncoder(items=500, width=64, q_heads=4, kv_heads=2, dim=64)
    for padding in (1, 63, 3000):
        cache = example.HistoryCache8(2, pages=1, kv_heads=2, page=16, dim=64, max_events=16, device="cuda")
        ids = torch.arange(1 + padding, dtype=torch.int32, device="cuda") % 500
        enc.step8(cache, i32([1]), ids, ids + 7, i32([1]), 1)
        assert cache.status.item() == 0 and cache.tables[1, 0] == 0
        assert cache.hours.tolist() == [7] + [0] * (cache.hours.numel() - 1)


def test_outputs_without_a_user_are_zero(example):  # noqa: F811
    """A call without room, and the padding of one that has it, beside memory that holds NaN."""
    enc = example.HistoryEncoder(items=500, width=64, q_heads=4, kv_heads=2, dim=64)
    cache = example.HistoryCache8(3, pages=4, kv_heads=2, page=16, dim=64, max_events=64, device="cuda")
    ids = torch.arange(70, dtype=torch.int32, device="cuda")
    for new, most, good in ((i32([33, 37]), 37, 0), (i32([16, 20]), 20, 36)):
        spoilt = [torch.full((70, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(8)]
        del spoilt
        out = enc.step8(cache, i32([2, 1]), ids, ids, new, most)
        assert cache.status.item() == (0 if good else example.ops.STATUS_NO_ROOM)
        assert torch.isfinite(out).all() and (out[good:] == 0).all() and (out[:good] != 0).any(1).all()
        cache.status.zero_()
