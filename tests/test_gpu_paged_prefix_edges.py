"""Attention of single tokens behind shared prefixes where it is easily wrong, on the GPU through the C ABI, against the
64-bit oracle.  Tolerances as in tests/test_gpu_paged_prefix.py.  A shared weight w of an e4m3 cache is rounded together
with its page's V scale s, as fp16 of w s 2^k with the largest such product W of the row at 2^7 or above when w is formed:
off by 2^-11 of it, or by half of fp16's smallest step, 2^-25 / 2^7 = 2^-32 of W, where that is more.  So a value's part
is off by at most |v| max(2^-11 w, 2^-32 W / s)."""
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


def _check_tails(made, q, out, scale):
    """As _check_attention without the lse, with the weights' rounding as the head of this file has it."""
    for i, t in enumerate(made.lens):
        for h in range(made.n_kv):
            k, v = made.held(i, h)
            ids = torch.tensor(made.rows[i], dtype=torch.long, device=DEV)[torch.arange(t, device=DEV) // made.P]
            s = made.c.v_scale[made.layer, ids, h].double()
            for g in range(made.G):
                qq = q[i, h * made.G + g].double()
                z = k @ qq * scale
                w = torch.softmax(z, dim=0)
                want, A = w @ v, w @ v.abs()
                big = float((k.abs() @ qq.abs() * abs(scale)).max())
                least = 2.0 ** -32 * (w * s).max() / s
                tol = 2.0 ** -8 * want.abs() + torch.maximum(2.0 ** -11 * w, least) @ v.abs() + (2 * 2.0 ** -17 * big + 2.0 ** -18) * A + 1e-30
                err = (out[i, h * made.G + g].double() - want).abs()
                assert bool(err.le(tol).all()), (i, h, g, float((err / tol).max()))


@pytest.mark.parametrize("gap", [6.0, 13.0, 16.0, 19.0, 25.0])
def test_long_flat_tails_behind_one_token(gap):
    """One shared token far above the others, whose value is 0 in half of the channels: there thousands of equal small
    weights alone make the result, down to those that fp16 has no number for."""
    made, prefix = _shared("e4m3", 16, 1, 2, [(20000, [20016 + 5 * i for i in range(3)])], 8)
    c, row = made.c, made.rows[0]
    c.k_pool[0, :, :, :, 0] = 0
    c.k_scale.fill_(0.125)
    c.v_scale.fill_(0.25)
    c.v_pool.view(torch.uint8)[0].bitwise_and_(0x7f)                                    # nothing cancels
    c.k_pool[0, row[40], 0, 7] = 0
    c.k_pool[0, row[40], 0, 7, 0] = torch.tensor(64.0, device=DEV).to(c.k_pool.dtype)
    c.v_pool[0, row[40], 0, 7, 64:] = 0
    q = torch.zeros(3, 2, 128, device=DEV)
    q[:, :, 0] = gap
    q[:, 1, 1] = 0.01
    q = q.to(torch.bfloat16)
    out = c.prefix_attn(0, K.PagedBatch(made.kv_len, made.table), prefix, q, scale=0.125)
    assert c.poll_error() == (0, 0)
    _check_tails(made, q, out, 0.125)


@pytest.mark.parametrize("down", [8, 16, 22, 40])
def test_values_of_pages_with_far_smaller_scales(down):
    """Pages of small values beside pages that have nothing in some channels: there the small ones alone count."""
    made, prefix = _shared("e4m3", 16, 1, 2, [(3000, [3008 + 5 * i for i in range(3)])], 8)
    c = made.c
    ids = torch.tensor(sorted({p for r in made.rows for p in r if p >= 0}), dtype=torch.long, device=DEV)
    c.v_pool.view(torch.uint8)[0].bitwise_and_(0x7f)
    fine = ids[::2]
    c.v_scale[0, ids] = 1.0
    c.v_scale[0, fine] = 2.0 ** -down
    c.v_pool.view(torch.uint8)[0, ids[1::2], :, :, 64:] = 0
    q = torch.randn(3, 2, 128, generator=_gen(2), device=DEV).to(torch.bfloat16)
    out = c.prefix_attn(0, K.PagedBatch(made.kv_len, made.table), prefix, q)
    assert c.poll_error() == (0, 0)
    _check_tails(made, q, out, 128 ** -0.5)
