"""The example's encoder end to end: histories appended event by event give the same outputs as in one
chunk, ranking stores nothing, and main() runs."""
import importlib.util
import os

import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    need_gpu()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "user_history.py")
    spec = importlib.util.spec_from_file_location("user_history", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_events_one_by_one_match_one_chunk(example):
    enc = example.HistoryEncoder(items=500, width=64, q_heads=6, kv_heads=2, dim=64, dtype=torch.float16)
    past = [37, 1, 20]
    make = lambda: example.HistoryCache(3, pages=16, kv_heads=2, page=16, dim=64, max_events=64, dtype=torch.float16, device="cuda")
    ids = [torch.randint(0, 500, (n,), dtype=torch.int32, generator=torch.Generator().manual_seed(n)).cuda() for n in past]
    hours = [torch.arange(n, device="cuda") * 3 for n in past]
    whole = make()
    out = enc.step(whole, [0, 1, 2], torch.cat(ids), torch.cat(hours), past).split(past)
    single = make()
    for i in range(max(past)):
        users = [u for u in range(3) if i < past[u]]
        got = enc.step(single, users, torch.stack([ids[u][i] for u in users]), torch.stack([hours[u][i] for u in users]),
                       [1] * len(users))
        for row, u in zip(got, users):
            # the same sums in another order: weights and result are each rounded to fp16 (2^-11 of values
            # below 8), the projection of another batch size may differ by one more such step in q, k and v
            assert (row - out[u][i]).abs().max() <= 8 * 4 * 2.0 ** -11
    assert single.held == whole.held == past


def test_ranking_stores_nothing_and_main_runs(example, capsys):
    enc = example.HistoryEncoder(items=500, width=64, q_heads=4, kv_heads=2, dim=64)
    cache = example.HistoryCache(2, pages=8, kv_heads=2, page=16, dim=64, max_events=64, dtype=torch.bfloat16, device="cuda")
    ids = torch.arange(30, dtype=torch.int32, device="cuda")
    enc.step(cache, [0, 1], ids, ids * 2, [20, 10])
    k, v = cache.k.clone(), cache.v.clone()
    a = enc.rank(cache, [1, 0], ids[:5], ids[:5] * 0 + 60, [2, 3])
    assert torch.equal(cache.k, k) and torch.equal(cache.v, v) and torch.isfinite(a).all()
    example.main()
    assert "best candidates" in capsys.readouterr().out
