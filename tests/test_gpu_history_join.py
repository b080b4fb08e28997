"""Long histories in many parts: both joins (a workgroup to a row where there are at most 512 rows and more than
16 parts, eight elements to a lane otherwise) after both attention kernels, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu
from history_util import History, np64
from sparse_embedding_lookup_dlrm_amd import ops
from test_gpu_history_attention import check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def parts_of(h, max_kv, causal=True, window=0):
    """Parts that the call is cut into, from the workspace it asks for."""
    N, Hq, D = h.q.shape
    need = ops.paged_attn_workspace_bytes(N, len(h.q_lens), Hq, h.k_cache.shape[1], D, causal, window, max(h.q_lens), max_kv)
    return need // (N * Hq * (4 * D + 8))


def run(h, window=0, causal=True):
    most = dict(max_q=max(h.q_lens), max_kv=max(h.kv_lens))
    got = check(h, causal=causal, window=window, **most)
    again = ops.paged_attn(*h.args(), causal=causal, window=window, want_lse=True, **most)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    return parts_of(h, max(h.kv_lens), causal, window)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("m", [1, 32])
def test_few_rows_many_parts(m, D, t):
    """8 rows (rows kernel) and 256 rows (tile kernel), at most 512: a workgroup joins a row."""
    assert run(History([m], [20_011], 8, 2, D, 16, t, seed=m + D)) > 16


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("D,Hq,Hk,q_lens,kv_lens", [
    (256, 16, 2, [1] * 40, [20_011] + [37 * i + 1 for i in range(39)]),  # rows kernel, 640 rows
    (64, 8, 2, [40, 3], [12_011, 5000]),                                 # tile kernel, 640 rows
    (128, 8, 2, [1, 40], [9000, 12_011])])
def test_many_rows_many_parts(D, Hq, Hk, q_lens, kv_lens, t):
    assert run(History(q_lens, kv_lens, Hq, Hk, D, 64, t, seed=D)) > 16


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("q_lens", [[1, 1, 1, 2], [20, 1, 3, 0]])
def test_long_and_short_histories_together(q_lens, t):
    """Parts of one history beside histories of one part, and without any entry."""
    h = History(q_lens, [40, 20_011, 0, 3000], 4, 1, 128, 32, t, seed=9)
    assert run(h) > 16
    run(h, causal=False)
    run(h, window=2500)


def test_as_many_parts_as_a_call_takes():
    """A history of 270,011 entries would be cut into 529 parts of 512; 511 is the most."""
    assert run(History([1], [270_011], 2, 1, 256, 128, "bf16", seed=4)) == 511


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("window", [0, 5000])
@pytest.mark.parametrize("D,group,m", [(64, 4, 3), (128, 2, 6), (64, 4, 40), (128, 4, 50), (256, 2, 60)])
def test_unseen_infinities_and_nan_in_parts(bad, window, D, group, m, t):
    """As with unsplit histories: what only later tokens see (with a window, also what only earlier ones see)
    reaches no other token."""
    held = 12_000 + m
    h, clean = (History([m], [held], 2 * group, 2, D, 16, t, seed=5) for _ in range(2))
    at = [12_000 + m // 2, held - 1] + ([12_000 - window + m // 3] if window else [])
    for e in at:
        pg = int(h.page_table[0, e // 16])
        h.v_cache[pg, 1, e % 16, 3::7] = bad
        h.k_cache[pg, 0, e % 16, 5] = bad
    got = ops.paged_attn(*h.args(), window=window, want_lse=True, max_q=m, max_kv=held)
    assert parts_of(h, held, window=window) > 1
    pos = np.arange(m) + 12_000
    untouched = np.ones(m, dtype=bool)
    for e in at:
        untouched &= ~((pos >= e) & (pos < e + window if window else True))
    if untouched.any():
        check(clean, window=window, got=got, rows=np.flatnonzero(untouched))
    assert ((~np.isfinite(np64(got[0])).all((1, 2))) == ~untouched).all()
