"""The example's page bookkeeping, which needs no GPU."""
import importlib.util
import os

import pytest
import torch


def make(**kw):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "user_history.py")
    spec = importlib.util.spec_from_file_location("user_history", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    how = dict(users=3, pages=6, kv_heads=1, page=16, dim=32, max_events=64, dtype=torch.bfloat16, device="cpu")
    how.update(kw)
    return m.HistoryCache(**how)


def test_histories_grow_by_pages():
    c = make()
    (offsets, lens, table), most = c.grow([0, 2], [17, 16])
    assert offsets.tolist() == [0, 17, 33] and lens.tolist() == [17, 16] and most == dict(max_q=17, max_kv=17)
    assert (table >= 0).sum(1).tolist() == [2, 1] and len(set(table[table >= 0].tolist())) == 3
    (_, lens, table), _ = c.grow([2], [1])
    assert lens.tolist() == [17] and (table >= 0).sum().item() == 2 and len(c.free) == 2


@pytest.mark.parametrize("users,new,match", [([0, 1], [1, 65], "room for 64"), ([1, 2], [17, 1], "2 are free"),
                                             ([1, 0, 1], [1, 1, 1], "one sequence")])
def test_without_room_nothing_changes(users, new, match):
    """A history longer than its row of the page table, more pages than are free, one user twice."""
    c = make()
    c.grow([0], [50])
    free, held, pages = list(c.free), list(c.held), [list(p) for p in c.pages]
    with pytest.raises(ValueError, match=match):
        c.grow(users, new)
    assert c.free == free and c.held == held and c.pages == pages
