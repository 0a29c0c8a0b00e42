"""Attention mass and eviction over the paged cache where they are easily wrong, on the GPU through the C ABI, against the
64-bit oracle.  Tolerances as in tests/test_gpu_paged_mass.py."""
import math

import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K
from compressed_kv_cache_vector_gb300.build import build
from tests.test_gpu_paged import Made, _gen, _i32
from tests.test_gpu_paged_mass import SCALE, _check_mass, _made_mass

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _cu(news):
    cu = [0]
    for x in news:
        cu.append(cu[-1] + x)
    return cu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [3, 128, 256, 257])
def test_queries_with_one_channel_far_above_the_others(kv, new):
    """A channel of 1000 beside others of 0.01, in which no key has anything: the others alone make the logits, however
    many rows the call has."""
    made = Made(kv, 32, 2, 1, [700, 300], 3)
    made.c.k_pool[..., 5] = 0
    if kv == "e4m3":
        made.c.k_scale.mul_(100)
    else:
        made.c.k_pool.mul_(100)
    news = [new, min(new, 77)]
    cu = _cu(news)
    q = 0.0101 * torch.randn(cu[-1], 2, 128, generator=_gen(2), device=DEV)
    q[..., 5] = 1000.0
    q = q.to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table, _i32(cu), new, cu[-1])
    _, lse = made.c.prefill_attn(0, b, q, lse=True)
    m = _made_mass(made, 2)
    before = m.mass.clone()
    made.c.prefill_mass(0, b, q, lse, m)
    assert made.c.poll_error() == (0, 0)
    _check_mass(made, before, m.mass, q, cu, news, SCALE, True, True, 0, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("news,G", [([20, 5, 1], 4), ([40, 5, 1], 4), ([100, 9, 64], 2), ([300, 70, 600], 4)])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_rows_without_a_sum_give_nothing(kv, news, G, what):
    """Rows whose lse is -infinity, single ones and whole tiles, with queries that are no numbers."""
    made = Made(kv, 16, 2, G, [900, 300, 700], 3)
    cu = _cu(news)
    q = torch.randn(cu[-1], 2 * G, 128, generator=_gen(2), device=DEV).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table, _i32(cu), max(news), cu[-1])
    _, lse = made.c.prefill_attn(0, b, q, lse=True)
    gone = torch.rand(lse.shape, generator=_gen(3), device=DEV) < 0.1
    gone[: min(50, cu[-1] // 2)] = True
    lse[gone] = -math.inf
    bad = q.clone()
    bad[gone] = what
    m = _made_mass(made, 2)
    before = m.mass.clone()
    made.c.prefill_mass(0, b, bad, lse, m)
    assert made.c.poll_error() == (0, 0)
    _check_mass(made, before, m.mass, q, cu, news, SCALE, True, True, 0, lse)
