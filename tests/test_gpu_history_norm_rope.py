"""Norm and rotation of queries and keys, their backward and the append to a paged cache, against
the fp64 oracle (tolerances: history_util)."""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu
from history_util import TYPES, U, History, Rope, close, half, norm_rope_tol, np64, rand, TINY
from oracle import history_oracle as ho
from sparse_embedding_lookup_dlrm_amd import ops

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _qkv(N, Hq, Hk, D, t, seed):
    """q, k, v as slices of one projection's output."""
    x = rand((N, (Hq + 2 * Hk) * D), t, seed)
    return x, Hq * D, (Hq + Hk) * D


def _split(x, Hq, Hk, D):
    N = x.shape[0]
    return (x[:, :Hq * D].view(N, Hq, D), x[:, Hq * D:(Hq + Hk) * D].view(N, Hk, D),
            x[:, (Hq + Hk) * D:].view(N, Hk, D))


# N, Hq, Hk, D, rot, axes, interleaved, norm
SHAPES = [(1, 1, 1, 32, 32, 1, False, True), (5, 8, 2, 64, 64, 1, False, True), (7, 3, 1, 64, 32, 2, True, True),
          (33, 12, 4, 128, 128, 3, False, False), (130, 2, 2, 256, 256, 2, True, True),
          (19, 5, 5, 128, 16, 1, False, True), (1030, 3, 1, 32, 16, 1, True, False),
          (2100, 4, 2, 128, 64, 1, False, True), (64, 1, 1, 256, 128, 3, True, True), (9, 2, 1, 64, 0, 1, False, True),
          (9000, 1, 1, 32, 32, 1, False, True)]


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(int(x)) for x in s))
def test_forward(shape, t):
    N, Hq, Hk, D, rot, axes, inter, norm = shape
    x, _, _ = _qkv(N, Hq, Hk, D, t, seed=N + D)
    r = Rope(N, D, rot, axes, norm, seed=N)
    pos, freq, w_q, w_k = r.dev()
    q, k, _ = _split(x.cuda(), Hq, Hk, D)
    qo, ko = ops.qk_norm_rope(q, k, pos, freq, w_q, w_k, eps=EPS, sections=r.sections, interleaved=inter)
    hq, hk, _ = _split(x, Hq, Hk, D)
    for got, src, w, name in ((qo, hq, r.w_q, "q"), (ko, hk, r.w_k, "k")):
        ref, mag = ho.norm_rope(np64(src), None if w is None else np64(w), r.angles(), inter, EPS)
        close(got, ref, norm_rope_tol(t, ref, mag), name)


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(int(x)) for x in s))
def test_backward(shape, t):
    N, Hq, Hk, D, rot, axes, inter, norm = shape
    x, _, _ = _qkv(N, Hq, Hk, D, t, seed=N + D)
    dq, dk = rand((N, Hq, D), t, 5), rand((N, Hk, D), t, 6)
    r = Rope(N, D, rot, axes, norm, seed=N)
    pos, freq, w_q, w_k = r.dev()
    q, k, _ = _split(x.cuda(), Hq, Hk, D)
    call = lambda: ops.qk_norm_rope_bwd(dq.cuda(), dk.cuda(), q, k, pos, freq, w_q, w_k, eps=EPS, sections=r.sections,
                                        interleaved=inter)
    got = call()
    hq, hk, _ = _split(x, Hq, Hk, D)
    for i, (dy, src, w, name) in enumerate(((dq, hq, r.w_q, "d_q"), (dk, hk, r.w_k, "d_k"))):
        dx, dw, mag, wmag = ho.norm_rope_bwd(np64(dy), np64(src), None if w is None else np64(w), r.angles(), inter, EPS)
        close(got[i], dx, half(t) * np.abs(dx) + 64 * U * mag + TINY[t], name)
        if norm:
            # each term is off by 64 u; the terms of a lane are added in a row, all of them at most
            close(got[2 + i], dw, (64 + src.shape[0] * src.shape[1]) * U * wmag, name + " weight")
        else:
            assert got[2 + i] is None
    again = call()  # the same bits
    for a, b in zip(got, again):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_gradient_against_differences():
    """The fp32 gradients along random directions against central differences of the fp64 forward:
    the difference quotient's own error is of order h^2 = 1e-8 of the terms' sizes."""
    N, Hq, Hk, D, rot = 6, 3, 2, 64, 32
    r = Rope(N, D, rot, 2, True, seed=4)
    q, k = rand((N, Hq, D), "f32", 1), rand((N, Hk, D), "f32", 2)
    dq, dk = rand((N, Hq, D), "f32", 3), rand((N, Hk, D), "f32", 4)
    pos, freq, w_q, w_k = r.dev()
    got = [np64(x) for x in ops.qk_norm_rope_bwd(dq.cuda(), dk.cuda(), q.cuda(), k.cuda(), pos, freq, w_q, w_k,
                                                  eps=EPS, sections=r.sections, interleaved=True)]
    rng = np.random.default_rng(0)
    for x, w, dy, gx, gw in ((q, r.w_q, dq, got[0], got[2]), (k, r.w_k, dk, got[1], got[3])):
        x, w, dy = np64(x), np64(w), np64(dy)
        loss = lambda x_, w_: (ho.norm_rope(x_, w_, r.angles(), True, EPS)[0] * dy).sum()
        for _ in range(5):
            ex, ew, h = rng.standard_normal(x.shape), rng.standard_normal(w.shape), 1e-4
            want = (loss(x + h * ex, w) - loss(x - h * ex, w)) / (2 * h)
            assert abs((gx * ex).sum() - want) <= 1e-5 * np.abs(gx * ex).sum() + 1e-5
            want = (loss(x, w + h * ew) - loss(x, w - h * ew)) / (2 * h)
            assert abs((gw * ew).sum() - want) <= 1e-5 * np.abs(gw * ew).sum() + 1e-5


def test_backward_takes_broadcast_gradients_and_no_tokens():
    D = 64
    r = Rope(8, D, 64, 1, True, seed=1)
    pos, freq, w_q, w_k = r.dev()
    q, k = rand((8, 4, D), "bf16", 1), rand((8, 2, D), "bf16", 2)
    one = rand((1, 1, D), "bf16", 3)
    a = ops.qk_norm_rope_bwd(one.cuda().expand(8, 4, D), one.cuda().expand(8, 2, D), q.cuda(), k.cuda(), pos, freq, w_q, w_k)
    b = ops.qk_norm_rope_bwd(one.cuda().expand(8, 4, D).contiguous(), one.cuda().expand(8, 2, D).contiguous(), q.cuda(),
                             k.cuda(), pos, freq, w_q, w_k)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    e = torch.empty((0, 4, D), dtype=torch.bfloat16, device="cuda")
    e2 = torch.empty((0, 2, D), dtype=torch.bfloat16, device="cuda")
    d_q, d_k, d_w_q, d_w_k = ops.qk_norm_rope_bwd(e, e2, e, e2, pos[:, :0], freq, w_q, w_k)
    assert d_q.shape == (0, 4, D) and not d_w_q.any() and not d_w_k.any()
    qo, ko = ops.qk_norm_rope(e, e2, pos[:, :0], freq, w_q, w_k)
    assert qo.shape == (0, 4, D) and ko.shape == (0, 2, D)


def test_far_and_negative_positions():
    """Angles of positions up to the ends of int32."""
    N, D = 64, 128
    g = torch.Generator().manual_seed(0)
    r = Rope(N, D, 128, 1, False, seed=0)
    r.positions = torch.randint(-2 ** 31, 2 ** 31 - 1, (1, N), generator=g).to(torch.int32)
    q, k = rand((N, 2, D), "f32", 1), rand((N, 1, D), "f32", 2)
    pos, freq, _, _ = r.dev()
    qo, _ = ops.qk_norm_rope(q.cuda(), k.cuda(), pos, freq)
    ref, mag = ho.norm_rope(np64(q), None, r.angles(), False, EPS)
    # 2^31 radians in fp64 are known to 2^-22 in the oracle too (its argument's rounding)
    close(qo, ref, norm_rope_tol("f32", ref, mag) + 2.0 ** -21 * mag, "q")


def test_strides_of_single_tokens_and_heads_are_not_looked_at():
    base = rand((5 * 64,), "bf16", 1).cuda()
    a = base.as_strided((5, 1, 64), (64, 3, 1))
    b = base.as_strided((1, 5, 64), (7, 64, 1))
    pos, freq = torch.arange(5, dtype=torch.int32, device="cuda"), torch.rand(32, device="cuda")
    qa, ka = ops.qk_norm_rope(a, a, pos, freq)
    qc, _ = ops.qk_norm_rope(a.contiguous(), a.contiguous(), pos, freq)
    assert torch.equal(qa, qc) and torch.equal(ka, qc)
    qb, _ = ops.qk_norm_rope(b, b, pos[:1], freq)
    assert torch.equal(qb, ops.qk_norm_rope(b.contiguous(), b.contiguous(), pos[:1], freq)[0])


def test_nan_and_infinity_stay_in_their_head():
    q, k = rand((4, 4, 64), "bf16", 1), rand((4, 2, 64), "bf16", 2)
    q[1, 2, 5], q[3, 0, 0] = float("nan"), float("inf")
    r = Rope(4, 64, 64, 1, True, seed=2)
    pos, freq, w_q, w_k = r.dev()
    qo, ko = ops.qk_norm_rope(q.cuda(), k.cuda(), pos, freq, w_q, w_k)
    fine = torch.isfinite(qo).all(-1).cpu()
    assert not fine[1, 2] and not fine[3, 0] and fine.sum() == 14 and torch.isfinite(ko).all()


# q_lens, kv_lens, Hq, Hk, D, page, rot, interleaved, norm
APPENDS = [([1], [1], 1, 1, 32, 16, 32, False, True), ([1] * 70, [(i * 37) % 200 + 1 for i in range(70)], 4, 2, 64, 16, 64, False, True),
           ([0, 5, 0, 33, 1, 0], [4, 5, 0, 70, 16, 9], 8, 2, 128, 32, 64, True, True),
           ([200, 1, 64], [500, 17, 64], 3, 3, 256, 64, 256, False, False),
           ([17, 18], [17, 40], 2, 1, 128, 128, 0, False, True)]


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("case", range(len(APPENDS)))
@pytest.mark.parametrize("with_q", [True, False])
def test_append(case, t, with_q):
    q_lens, kv_lens, Hq, Hk, D, page, rot, inter, norm = APPENDS[case]
    h = History(q_lens, kv_lens, Hq, Hk, D, page, t, seed=case)
    N = sum(q_lens)
    x, _, _ = _qkv(N, Hq, Hk, D, t, seed=9)
    r = Rope(N, D, rot, 2 if rot else 1, norm, seed=case)
    pos, freq, w_q, w_k = r.dev()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, v = _split(x.cuda(), Hq, Hk, D)
    _, kc, vc, off, lens, table = h.args()
    qo = ops.kv_append(k, v, kc, vc, off, lens, table, q=q if with_q else None, positions=pos if rot else None,
                       inv_freq=freq, w_q=w_q if with_q else None, w_k=w_k, eps=EPS,
                       sections=r.sections if rot else None, interleaved=inter, status=status)
    assert status.item() == 0
    hq, hk, hv = _split(x, Hq, Hk, D)
    if with_q:
        ref, mag = ho.norm_rope(np64(hq), None if not norm else np64(r.w_q), r.angles(), inter, EPS)
        close(qo, ref, norm_rope_tol(t, ref, mag), "q")
    else:
        assert qo is None
    ref, mag = ho.norm_rope(np64(hk), None if not norm else np64(r.w_k), r.angles(), inter, EPS)
    tol = norm_rope_tol(t, ref, mag)
    want_k, want_v, touched = h.k_cache.clone(), h.v_cache.clone(), torch.zeros(h.k_cache.shape[0], page, dtype=torch.bool)
    kc, vc = kc.cpu(), vc.cpu()
    for n, at in enumerate(ho.slots(h.q_offsets.tolist(), kv_lens, h.page_table.tolist(), page, kc.shape[0])):
        close(kc[at[0], :, at[1]], ref[n], tol[n], f"k of token {n}")
        assert torch.equal(vc[at[0], :, at[1]], hv[n])
        touched[at[0], at[1]] = True
    keep = ~touched[:, None, :, None].expand_as(kc)
    bits = lambda c: c.view(torch.int16)
    assert torch.equal(bits(kc)[keep], bits(want_k)[keep]) and torch.equal(bits(vc)[keep], bits(want_v)[keep])


def test_append_reports_bad_pages_and_lengths_and_stores_the_rest():
    Hk, D, page = 2, 64, 16
    h = History([3, 2, 4, 2], [20, 30, 2, 40], 2, Hk, D, page, "bf16", seed=3)
    q, kc, vc, off, lens, table = h.args()
    N = q.shape[0]
    k, v = rand((N, Hk, D), "bf16", 1), rand((N, Hk, D), "bf16", 2)
    table[0, 1] = kc.shape[0]   # past the last page
    lens[3] = 10 ** 6           # past the page table
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc0, vc0 = kc.clone(), vc.clone()
    ops.kv_append(k.cuda(), v.cuda(), kc, vc, off, lens, table, status=status)
    assert status.item() == ops.STATUS_BAD_PAGE | ops.STATUS_BAD_OFFSETS
    pages = table.cpu()
    stored = {3: (1, 28), 4: (1, 29), 7: (2, 0), 8: (2, 1)}  # sequence 2 holds 2 of its 4 tokens
    bits = lambda x: x.view(torch.int16)
    for n, (s, at) in stored.items():
        pg = int(pages[s, at // page])
        assert torch.equal(kc[pg, :, at % page].cpu(), k[n]) and torch.equal(vc[pg, :, at % page].cpu(), v[n])
        kc[pg, :, at % page] = kc0[pg, :, at % page]
        vc[pg, :, at % page] = vc0[pg, :, at % page]
    assert torch.equal(bits(kc), bits(kc0)) and torch.equal(bits(vc), bits(vc0))


def test_append_into_a_layer_of_a_larger_cache_and_padded_tokens():
    """The caches as slices of [pages, layers, heads, page, dim]; tokens past the last sequence are not stored."""
    Hk, D, page = 2, 64, 16
    big_k = torch.zeros((6, 3, Hk, page, D), dtype=torch.float16, device="cuda")
    big_v = torch.zeros_like(big_k)
    k, v = rand((5, Hk, D), "f16", 1).cuda(), rand((5, Hk, D), "f16", 2).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ops.kv_append(k, v, big_k[:, 1], big_v[:, 1], i32([0, 1, 3]), i32([17, 2]), i32([[4, 2], [5, 0]]))
    for at, n in (((2, 1, slice(None), 0), 0), ((5, 1, slice(None), 0), 1), ((5, 1, slice(None), 1), 2)):
        assert torch.equal(big_k[at], k[n]) and torch.equal(big_v[at], v[n])
        big_k[at], big_v[at] = 0, 0
    assert not big_k.any() and not big_v.any()


def test_backward_of_more_than_the_caches_hold():
    """Inputs past 256 MB are read another way: the same bits as the same tokens in two smaller calls, the
    weight gradients the sum of theirs."""
    N, Hq, Hk, D = 16384, 32, 8, 128
    g = torch.Generator("cuda").manual_seed(0)
    q, dq = (torch.randn((N, Hq, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    k, dk = (torch.randn((N, Hk, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    r = Rope(N, D, 128, 1, True, seed=0)
    pos, freq, w_q, w_k = r.dev()
    whole = ops.qk_norm_rope_bwd(dq, dk, q, k, pos, freq, w_q, w_k)
    a, b = (ops.qk_norm_rope_bwd(dq[c], dk[c], q[c], k[c], pos[:, c], freq, w_q, w_k)
            for c in (slice(0, N // 2), slice(N // 2, N)))
    for i in (0, 1):
        assert torch.equal(whole[i], torch.cat([a[i], b[i]]))
    for i, many in ((2, N * Hq), (3, N * Hk)):
        # each side is off by a few u of the sum of sizes, about many; lanes add at most 64 terms in a row
        assert ((whole[i] - a[i] - b[i]).abs() <= 2 * 80 * U * many).all()
