"""Pages handed out and taken back on the device against the oracle, which hands them out one by one. All results
are whole numbers and have to be equal."""
import random

import pytest
import torch

from gpu_util import need_gpu
from oracle import history_oracle as ho
from sparse_embedding_lookup_dlrm_amd import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class State:
    def __init__(self, users, width, page, held, seed, spare=50):
        rng = random.Random(seed)
        self.page = page
        self.held = list(held)
        need = [-(-h // page) for h in self.held]
        total = sum(need) + spare
        order = list(range(total))
        rng.shuffle(order)
        self.tables = [[-7] * width for _ in range(users)]
        for u, m in enumerate(need):
            self.tables[u][:m] = [order.pop() for _ in range(m)]
        self.count = len(order)
        self.free = order + [-9] * (total - len(order))
        self.width = width
        self.dev()

    def dev(self):
        self.d = (i32(self.held), i32(self.tables).reshape(len(self.held), self.width), i32(self.free), i32([self.count]))

    def same(self, held, tables=None, free=None, count=None):
        assert self.d[0].tolist() == held
        if tables is not None:
            for u, row in enumerate(self.d[1].tolist()):
                m = -(-min(max(held[u], 0), self.width * self.page) // self.page)
                assert row[:m] == tables[u][:m], u
        assert free is None or self.d[2].tolist() == free
        assert self.d[3].item() == count
        self.held, self.count = held, count
        self.tables = self.tables if tables is None else tables
        self.free = self.free if free is None else free

    def assign(self, new, users, N=None, width=None, **kw):
        N = sum(max(m, 0) for m in new) if N is None else N
        width = self.width if width is None else width
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = ops.pages_assign(i32(new), *self.d, self.page, N, users=None if users is None else i32(users), table_width=width,
                               status=status, **kw)
        bits, want, state = ho.pages_assign(new, range(len(new)) if users is None else users, self.held, self.tables, self.free,
                                            self.count, self.page, N, width)
        assert status.item() == bits
        for name, g, w in zip(("q_offsets", "kv_lens", "page_table", "slots", "positions"), got, want):
            assert g.tolist() == w, name
        assert got[3].dtype == torch.int64
        return bits, state

    def release(self, users, keep=None):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.pages_release(*self.d, self.page, users=None if users is None else i32(users), keep=None if keep is None else i32(keep),
                          status=status)
        who = range(len(self.held)) if users is None else users
        bits, held, free, count = ho.pages_release(who, [0] * len(who) if keep is None else keep, self.held, self.tables, self.free,
                                                   self.count, self.page)
        assert status.item() == bits
        self.same(held, free=free, count=count)
        return bits


@pytest.mark.parametrize("page", [16, 64, 65536])
@pytest.mark.parametrize("seqs,most", [(1, 1), (1, 5000), (3, 40), (64, 1), (65, 33), (1024, 3), (1025, 40), (3001, 2)])
def test_assign_then_release(seqs, most, page):
    rng = random.Random(seqs * most + page)
    users = seqs + rng.randint(0, 20)
    held = [rng.choice([0, 1, page - 1, page, rng.randint(0, 200)]) for _ in range(users)]
    width = max(-(-(h + 3 * most) // page) for h in held) + 1
    st = State(users, width, page, held, seed=seqs, spare=3 * (seqs + seqs * most // page) + 5)
    who = rng.sample(range(users), seqs)
    for step in range(3):
        new = [rng.randint(0, most) for _ in range(seqs)]
        bits, state = st.assign(new, who, N=sum(new) + rng.choice([0, 1, 700]))
        assert bits == 0
        st.same(*state[:2], count=state[2])
    assert st.release(who, [rng.randint(0, st.held[u] + 2) for u in who]) == 0
    assert st.release(None) == 0
    assert not any(st.held) and sorted(st.free[:st.count]) == list(range(len(st.free)))


def test_without_users_and_with_a_narrow_table():
    st = State(5, 9, 16, [0, 16, 17, 3, 40], seed=1)
    bits, state = st.assign([1, 16, 0], None, width=3)
    assert bits == 0
    st.same(*state[:2], count=state[2])
    bits, state = st.assign([0, 0, 0, 0, 0], None)  # nothing new: the tables of the histories as they are
    assert bits == 0 and st.d[0].tolist() == st.held


def test_none_and_no_sequences():
    st = State(3, 4, 16, [5, 0, 20], seed=1)
    off, lens, table, slots, places = ops.pages_assign(i32([]), *st.d, 16, 3, users=i32([]))
    assert off.tolist() == [0] and lens.numel() == 0 and table.shape == (0, 4)
    assert slots.tolist() == [-1] * 3 and places.tolist() == [-1] * 3
    got = ops.pages_assign(i32([1, 0]), *st.d, 16, 5, want_slots=False)
    assert got[3] is None and got[4] is None and st.d[0].tolist() == [6, 0, 20]
    ops.pages_release(*st.d, 16, users=i32([]))
    assert st.d[0].tolist() == [6, 0, 20]


REFUSED = [
    (dict(new=[1, 1, 1], users=[0, 9, 1]), ops.STATUS_BAD_USER),
    (dict(new=[1, 1, 1], users=[0, -1, 1]), ops.STATUS_BAD_USER),
    (dict(new=[1, 1, 1], users=[2, 0, 2]), ops.STATUS_BAD_USER),
    (dict(new=[1, -1, 1], users=[0, 1, 2]), ops.STATUS_BAD_OFFSETS),
    (dict(new=[4, 4, 4], users=[0, 1, 2], N=11), ops.STATUS_BAD_OFFSETS),
    (dict(new=[2 ** 31 - 1, 2 ** 31 - 1, 5], users=[0, 1, 2], N=100), ops.STATUS_BAD_OFFSETS | ops.STATUS_NO_ROOM),
    (dict(new=[1, 1, 100], users=[0, 1, 2]), ops.STATUS_NO_ROOM),
    (dict(new=[1, 1, 1], users=[0, 1, 2], width=1), ops.STATUS_NO_ROOM),
    (dict(new=[60, 60, 40], users=[0, 1, 3]), ops.STATUS_NO_ROOM),  # too few pages
    (dict(new=[1, 1, 1], users=[0, 1, 4]), ops.STATUS_BAD_OFFSETS),  # a user's length is negative
    (dict(new=[1, 1, 1], users=[0, 1, 5]), ops.STATUS_BAD_OFFSETS),  # or past its table
]


@pytest.mark.parametrize("kw,bits", REFUSED)
def test_refused_calls_change_nothing(kw, bits):
    st = State(6, 5, 16, [0, 16, 37, 3, 0, 0], seed=4, spare=7)
    st.held[4], st.held[5] = -3, 81
    st.dev()
    before = [x.clone() for x in st.d]
    got, state = st.assign(**kw)
    assert got == bits
    for a, b in zip(before, st.d):
        assert torch.equal(a, b)


@pytest.mark.parametrize("count", [-1, 100])
def test_bad_free_count(count):
    st = State(3, 5, 16, [0, 16, 37], seed=4, spare=7)
    st.count = count
    st.dev()
    # fewer than none are too few as well
    assert st.assign([1, 1], [0, 2])[0] == ops.STATUS_BAD_PAGE | (ops.STATUS_NO_ROOM if count < 0 else 0)
    assert st.release([0, 2]) == ops.STATUS_BAD_PAGE and st.d[3].item() == count


@pytest.mark.parametrize("users,keep,bits", [([0, 9], [0, 0], 16), ([0, 2, 0], [0, 0, 0], 16), ([0, 2], [0, -1], 2), ([4, 2], [0, 0], 2),
                                             ([2, 1], [0, 0], 4)])
def test_refused_releases_change_nothing(users, keep, bits):
    st = State(5, 5, 16, [0, 16, 37, 3, 0], seed=4, spare=7)
    st.held[4] = 81
    if bits == 4:  # the list is fuller than it can be
        st.count += 2
    st.dev()
    before = [x.clone() for x in st.d]
    assert st.release(users, keep) == bits
    for a, b in zip(before, st.d):
        assert torch.equal(a, b)


def test_a_user_twice_without_new_entries():
    """Candidates of one user in two sequences, beside new entries in a third: all see the history as it was."""
    st = State(3, 5, 16, [10, 16, 37], seed=4)
    bits, state = st.assign([0, 5, 0, 0], [2, 2, 2, 1])
    assert bits == 0
    st.same(*state[:2], count=state[2])


def test_bad_pages_in_a_users_row():
    st = State(2, 5, 16, [10, 20], seed=4)
    st.tables[0][0], st.tables[1][0] = -5, 10 ** 6
    st.dev()
    bits, state = st.assign([3, 3], None)
    assert bits == ops.STATUS_BAD_PAGE
    st.same(*state[:2], count=state[2])


def test_planned_steps_leave_the_state():
    st = State(40, 30, 16, [i * 7 for i in range(40)], seed=4, spare=90)
    held, count = torch.full_like(st.d[0], -1), torch.full_like(st.d[3], -1)
    for _ in range(2):
        bits, state = st.assign([3] * 20, list(range(0, 40, 2)), held_out=held, count_out=count)
        assert bits == 0 and st.d[0].tolist() == st.held and st.d[3].item() == st.count
        assert held.tolist() == [state[0][u] if u % 2 == 0 else -1 for u in range(40)] and count.item() == state[2]
    back, more = torch.zeros_like(held), torch.zeros_like(count)
    ops.pages_release(*st.d, 16, users=i32([3, 39]), held_out=back, count_out=more)
    assert st.d[0].tolist() == st.held and st.d[3].item() == st.count
    assert not back.any() and more.item() == st.count + 2 + 18


def test_strided_tables_another_stream_and_graph_replays():
    st = State(20, 8, 16, [i * 3 for i in range(20)], seed=5, spare=300)
    wide = torch.full((20, 13), -7, dtype=torch.int32, device="cuda")
    wide[:, 2:10] = st.d[1]
    st.d = (st.d[0], wide[:, 2:10], *st.d[2:])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    new, users = [2, 0, 19], [4, 5, 19]
    with torch.cuda.stream(s):
        bits, state = st.assign(new, users)
    assert bits == 0
    torch.cuda.current_stream().wait_stream(s)
    st.same(*state[:2], count=state[2])
    assert (wide[:, :2] == -7).all() and (wide[:, 10:] == -7).all()

    new_d, who = i32([1, 1, 1]), i32([0, 1, 2])
    keep = i32([0, 3, 6])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = ops.pages_assign(new_d, *st.d, 16, 10, users=who)
        ops.pages_release(*st.d, 16, users=who, keep=keep)
    for i in range(4):
        new = [i + 1, 0, 3]
        new_d.copy_(i32(new))
        bits, want, (held, tables, count) = ho.pages_assign(new, [0, 1, 2], st.held, st.tables, st.free, st.count, 16, 10, 8)
        graph.replay()
        torch.cuda.synchronize()
        assert bits == 0
        for g, w in zip(got, want):
            assert g.tolist() == w
        bits, held, free, count = ho.pages_release([0, 1, 2], [0, 3, 6], held, tables, st.free, count, 16)
        st.same(held, free=free, count=count)


def test_one_long_history():
    """A history of more than a million entries, more than one launch dimension of sequences beside it."""
    U = 70_001
    page, width = 16, 66_000
    held = torch.zeros(U, dtype=torch.int32, device="cuda")
    base = torch.full((width,), -1, dtype=torch.int32, device="cuda")
    # one row for all users but the last: those get one page, so their rows may not overlap
    tables = torch.full((U, 1), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(2 * U, device="cuda").to(torch.int32)
    count = i32([2 * U])
    new = torch.ones(U, dtype=torch.int32, device="cuda")
    off, lens, table, slots, places = ops.pages_assign(new, held, tables, free, count, page, U)
    assert torch.equal(off.long(), torch.arange(U + 1, device="cuda")) and (lens == 1).all() and (places == 0).all()
    assert torch.equal(table[:, 0], free.flip(0)[:U]) and torch.equal(slots, table[:, 0].long() * page) and count.item() == U
    held, tables = i32([7]), base[None].clone()
    tables[0, 0] = 3
    free = torch.arange(70_000, dtype=torch.int32, device="cuda")
    N = 1_050_000
    off, lens, table, slots, places = ops.pages_assign(i32([N]), held, tables, free, i32([70_000]), page, N + 10)
    e = torch.arange(7, 7 + N, device="cuda")
    pages = torch.where(e < 16, torch.full_like(e, 3), 70_000 - (e // 16))
    assert off.tolist() == [0, N] and torch.equal(places[:N].long(), e) and torch.equal(slots[:N], pages * 16 + e % 16)
    assert (slots[N:] == -1).all() and (places[N:] == -1).all()


@pytest.mark.parametrize("a,b", [(5, 2900), (5, 5 + 1024), (0, 2999), (63, 64), (1023, 1024)])
def test_a_user_twice_far_apart(a, b):
    """In sequences that different lanes, waves and turns of the deciding workgroup look at."""
    users = 3100
    st = State(users, 4, 16, [u % 30 for u in range(users)], seed=9, spare=6000)
    who = list(range(50, 3050))
    assert st.assign([1] * 3000, who)[0] == 0
    st.held = st.d[0].tolist()
    st.tables, st.count = st.d[1].tolist(), st.d[3].item()
    who[b] = who[a]
    before = [x.clone() for x in st.d]
    assert st.assign([1] * 3000, who)[0] == ops.STATUS_BAD_USER
    assert st.release(who) == ops.STATUS_BAD_USER
    for x, y in zip(before, st.d):
        assert torch.equal(x, y)


def test_lengths_that_are_the_state_are_refused():
    """All entries kept, and every history doubled, by the tensor of the lengths themselves: refused, nothing changes; a
    copy does it."""
    st = State(5, 9, 16, [0, 16, 17, 3, 40], seed=1)
    before = [x.clone() for x in st.d]
    with pytest.raises(ops.DlrmError):
        ops.pages_release(*st.d, 16, keep=st.d[0])
    with pytest.raises(ops.DlrmError):
        ops.pages_assign(st.d[0], *st.d, 16, 200)
    with pytest.raises(ops.DlrmError):
        ops.pages_release(*st.d, 16, users=st.d[0][:1])
    for a, b in zip(before, st.d):
        assert torch.equal(a, b)
    assert st.release(None, st.held) == 0
    bits, state = st.assign(st.held, None)
    assert bits == 0
    st.same(*state[:2], count=state[2])


@pytest.mark.parametrize("bad", [-5, 10 ** 6, 46])
@pytest.mark.parametrize("seqs,at", [(1, 0), (3, 2), (70, 1), (70, 2500), (1100, 7)])
def test_a_bad_page_is_not_released(bad, seqs, at):
    """A page outside the cache among those that would go back: the call is refused, in place and planned, whichever
    workgroup meets it; it goes back without its user, or where the user keeps it."""
    rng = random.Random(seqs + at)
    users = seqs + 3
    held = [rng.randint(1, 60) for _ in range(users)]
    user = seqs // 2
    held[user] = 16 * at + rng.randint(1, 16)
    width = at + 6
    st = State(users, width, 16, held, seed=seqs, spare=30)
    bad = len(st.free) if bad == 46 else bad  # the first that does not exist
    good = st.tables[user][at]
    st.tables[user][at] = bad
    st.dev()
    who = rng.sample([u for u in range(users) if u != user], seqs - 1)
    who.insert(seqs // 3, user)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = [x.clone() for x in st.d]
    other, more = torch.full_like(st.d[0], -1), torch.full_like(st.d[3], -1)
    for keep in (None, [16 * at if u == user else rng.randint(0, 9) for u in who]):
        for kw in (dict(held_out=other, count_out=more), {}):
            ops.pages_release(*st.d, 16, users=i32(who), keep=None if keep is None else i32(keep), status=status, **kw)
            assert status.item() == ops.STATUS_BAD_PAGE
            status.zero_()
            assert torch.equal(before[0], st.d[0]) and torch.equal(before[1], st.d[1]) and torch.equal(before[3], st.d[3])
            assert torch.equal(before[2][:st.count], st.d[2][:st.count])
        assert more.item() == st.count and all(other[u] == held[u] for u in who)
    bits, want = ho.pages_release(who, [0] * seqs, st.held, st.tables, st.free, st.count, 16)[:2]
    assert bits == ops.STATUS_BAD_PAGE and want == st.held
    # kept: the rest goes back
    st.free = st.d[2].tolist()
    assert st.release(who, [16 * at + 1 if u == user else 0 for u in who]) == 0
    st.tables[user][at] = good
    st.d[1][user, at] = good
    assert st.release(None) == 0 and sorted(st.free) == list(range(len(st.free)))
