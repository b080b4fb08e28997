"""Limits of the user-history operators' sizes, which need no GPU: refused before any HIP call."""
import ctypes

import pytest

from sparse_embedding_lookup_dlrm_amd import ops
from test_history_abi import E_UNSUPPORTED, _append, _attn


@pytest.fixture(scope="module")
def lib():
    return ops.lib()


def test_more_sequences_than_a_counter_holds_are_refused(lib):
    """Kernels count sequences in 32 bits, in steps of up to 65535, and search their offsets in blocks."""
    for S in (2 ** 31 - 2, 2 ** 31 - 65536, 2 ** 31 - (1 << 17)):
        assert _attn(lib, S=S) == E_UNSUPPORTED and _append(lib, S=S) == E_UNSUPPORTED, S
        need = ctypes.c_size_t(0)
        assert lib.dlrm_paged_attn_workspace_bytes(4, S, 4, 2, 64, 1, 0, 2, 128, ctypes.byref(need)) == E_UNSUPPORTED
