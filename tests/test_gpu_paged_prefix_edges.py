"""Attention of single tokens behind shared prefixes where it is easily wrong, on the GPU through the C ABI, against the
64-bit oracle.  Tolerances as in tests/test_gpu_paged_prefix.py."""
import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K
from compressed_kv_cache_vector_gb300.build import build
from tests.test_gpu_paged import _check_attention, _gen
from tests.test_gpu_paged_prefix import ROUND, _shared

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_queries_with_one_channel_far_above_the_others(kv):
    """A channel of 1000 beside others of 0.01, in which no key has anything: the others alone make the logits."""
    made, prefix = _shared(kv, 32, 2, 4, [(900, [950, 901, 900, 1200]), (300, [340, 300])], 8)
    made.c.k_pool[..., 5] = 0
    if kv == "e4m3":
        made.c.k_scale.mul_(100)
    else:
        made.c.k_pool.mul_(100)
    q = 0.0101 * torch.randn(6, 8, 128, generator=_gen(2), device=DEV)
    q[..., 5] = 1000.0
    q = q.to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table)
    out, lse = made.c.prefix_attn(0, b, prefix, q, lse=True)
    assert made.c.poll_error() == (0, 0)
    _check_attention(made, q, out, lse, 128 ** -0.5, [1] * 6, True, ROUND[kv])
