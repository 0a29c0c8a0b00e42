"""The tests of tests/test_gpu_paged_prefix.py again with page tables twice as wide, so that no batch of theirs is small
enough for its sequences to read what they share each by themselves; and where that border lies."""
import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K
from tests import test_gpu_paged_prefix as P
from tests.test_gpu_paged import Made, _gen, _i32
from tests.test_gpu_paged_prefix import (  # noqa: F401
    _built, test_a_nan_key_reaches_the_rows_that_see_it, test_captured_with_groups_that_change,
    test_groups_of_every_shape, test_many_groups_of_long_prefixes, test_more_cells_than_runs,
    test_one_shared_token_with_nearly_all_weight, test_rows_of_every_number,
    test_rows_strided_padded_absent_and_on_a_stream, test_scales_and_growing_logits, test_v_scales_far_apart,
    test_wrong_groups_share_nothing_and_are_told)

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _wider(monkeypatch):
    monkeypatch.setattr(P, "Made", lambda *a, extra_cols=2, **k: Made(*a, extra_cols=2 * extra_cols, **k))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("mib,shares", [(100, False), (144, False), (145, True)])
def test_border_of_small_batches(kv, mib, shares):
    """Up to 144 MiB that the table could name, decode_attn's results to the bit; beyond, the groups' pages are shared."""
    n, page, n_kv = 8, 32, 2
    columns = mib * 2 ** 20 // (n * page * n_kv * 256 * (1 if kv == "e4m3" else 2))
    made = Made(kv, page, n_kv, 4, [3000 + 7 * i for i in range(n)], 3, extra_cols=0)
    table = torch.full((n, columns), -7, dtype=torch.int32, device=DEV)
    table[:, :made.table.shape[1]] = made.table
    table[:, :90] = made.table[0, :90]
    assert columns * n * page * n_kv * 256 * (1 if kv == "e4m3" else 2) == mib * 2 ** 20
    q = torch.randn(n, 8, 128, generator=_gen(2), device=DEV).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, table)
    out, lse = made.c.prefix_attn(0, b, K.PagedPrefix(_i32([0, n]), _i32([2880])), q, lse=True)
    ref, ref_lse = made.c.decode_attn(0, b, q, lse=True)
    assert made.c.poll_error() == (0, 0)
    assert (torch.equal(out, ref) and torch.equal(lse, ref_lse)) != shares
