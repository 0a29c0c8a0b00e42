"""Eviction from the paged cache where it is easily wrong, on the GPU through the C ABI, against the definition."""
import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K
from compressed_kv_cache_vector_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


@pytest.mark.parametrize("cut", [True, False])
def test_longest_sequence_that_a_table_can_name(cut):
    """2^31 - 256 tokens behind a prefix that is one page over and over: the last page's one free choice is cut, or
    nothing is."""
    P, columns = 64, (2 ** 31 - 256) // 64
    T = columns * P
    c = K.PagedKV(K.make_paged_config(1, 1, 1, P, 3, 1, K.MK_KV_E4M3), DEV)
    c.k_pool.view(torch.uint8).copy_(torch.randint(0, 120, c.k_pool.shape, dtype=torch.uint8, device=DEV))
    c.v_pool.view(torch.uint8).copy_(torch.randint(0, 120, c.v_pool.shape, dtype=torch.uint8, device=DEV))
    c.k_scale.fill_(2.0 ** 20)                                                          # so that a page's scale is formed anew
    c.v_scale.fill_(2.0 ** 20)
    table = torch.zeros(1, columns, dtype=torch.int32, device=DEV)
    table[0, -1] = 2
    m = K.PagedMass(c)
    before = [t.clone() for t in (c.k_pool.float(), c.v_pool.float())]
    keep = T - 1 if cut else T
    new_len, kept = c.evict(0, K.PagedBatch(torch.tensor([T], dtype=torch.int32, device=DEV), table), m,
                            torch.tensor([keep], dtype=torch.int32, device=DEV), first=T - 2, recent=1, max_keep=keep)
    assert c.poll_error() == (0, 0) and new_len.tolist() == [keep]
    step = 1 << 28
    for a in range(0, keep - cut, step):
        e = min(keep - cut, a + step)
        assert torch.equal(kept[0, 0, a:e], torch.arange(a, e, dtype=torch.int32, device=DEV))
    for t, was, scale in ((c.k_pool, before[0], c.k_scale), (c.v_pool, before[1], c.v_scale)):
        now = t.float() * scale[..., None, None]
        assert torch.equal(now[0, :2], was[0, :2] * 2.0 ** 20)                           # the pages of the prefix, and one of nobody
        assert torch.equal(now[0, 2, 0, :62], was[0, 2, 0, :62] * 2.0 ** 20)
        assert torch.equal(now[0, 2, 0, 62], was[0, 2, 0, 63 if cut else 62] * 2.0 ** 20)
    if cut:
        assert int(kept[0, 0, -1]) == T - 1
