"""What the paged cache's workspace holds, from its sizes (on the CPU)."""
import ctypes

import pytest

from compressed_kv_cache_vector_gb300 import binding as K
from compressed_kv_cache_vector_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return K.load()


def _bytes(lib, n_pages=100, max_seqs=16, n_q=32, n_kv=8, page=32):
    w = ctypes.c_size_t()
    cfg = K.make_paged_config(n_q, n_kv, 2, page, n_pages, max_seqs, K.MK_KV_E4M3)
    assert lib.mk_paged_sizes(ctypes.byref(cfg), None, None, ctypes.byref(w)) == 0
    return w.value


def test_prefixes_steps_with_mass_and_eviction_take_turns(lib):
    """Two parts of 528 bytes a sequence and query head (prefixes), or two words a page and kv head (eviction): the
    larger of them, not both."""
    rows = 2 * 528 * 256 * 64
    few, many = (_bytes(lib, n_pages=n, max_seqs=256, n_q=64) for n in (10, 100000))
    assert few == many and 8 * 100000 * 8 < rows                                        # the rows' parts hold it
    big = _bytes(lib, n_pages=1000000, max_seqs=256, n_q=64)
    assert abs(big - few - (8 * 1000000 * 8 - rows)) < 1 << 17                           # the groups, the plan and the words beside the parts
