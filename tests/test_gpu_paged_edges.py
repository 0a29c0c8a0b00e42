"""The paged cache where a call meets a limit of its kernels: contexts so long that waits inside a kernel last, numbers
that are not finite, scales far apart, errors of one sequence beside good ones, lengths that go back.

The bounds are those of test_gpu_paged.py; a test that needs another one derives it beside its inputs.
"""
import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K
from compressed_kv_cache_vector_gb300.build import build
from oracle import paged_oracle as O
from tests.test_gpu_paged import DEV, KV, _gen, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_chunk_behind_a_million_tokens_whose_last_row_tile_is_narrow(kv):
    """4100 new tokens of 1,048,576: the last row tile has 4 tokens (16 rows), so a CTA runs several items of one row
    tile and 8192 steps each, some 50 ms, while the warps of the other row tile wait for the next item of two.

    The sums of a row are of up to N = 8 x 8192 terms one after the other, in the softmax as in the products: off by at
    most N / 2 x 2^-24 = 2^-9 of their size, and the products' additions, which may cut off, by 2^-8 of the weighted
    |v|, on top of test_gpu_paged.py's bounds."""
    T, m, P, n_kv, G = 1 << 20, 4100, 64, 8, 4
    n_pages, g = T // P + 3, _gen(1)
    c = K.PagedKV(K.make_paged_config(n_kv * G, n_kv, 1, P, n_pages, 1, KV[kv]), DEV)
    for pool in (c.k_pool, c.v_pool):
        for a in range(0, n_pages, 1024):
            y = torch.randn(min(1024, n_pages - a), n_kv, P, 128, generator=g, device=DEV)
            pool[0, a:a + 1024] = (y * 64 if kv == "e4m3" else y).to(pool.dtype)
    if kv == "e4m3":
        c.k_scale.fill_(2.0 ** -6)
        c.v_scale.fill_(2.0 ** -6)
    ids = torch.randperm(n_pages, generator=g, device=DEV)[: T // P]
    q = (4 * torch.randn(m, n_kv * G, 128, generator=g, device=DEV)).to(torch.bfloat16)
    b = K.PagedBatch(_i32([T]), ids.int()[None].contiguous(), _i32([0, m]), m, m)
    out, lse = c.prefill_attn(0, b, q, lse=True)
    assert c.poll_error() == (0, 0)
    rows = torch.tensor([0, 63, 2049, 4095, 4096, 4099], device=DEV)
    for h in (0, 3, 7):
        k, v = ((p[0, :, h].view(torch.uint8 if kv == "e4m3" else torch.int16)[ids].view(p.dtype).double()
                 * (2.0 ** -6 if kv == "e4m3" else 1.0)).reshape(T, 128) for p in (c.k_pool, c.v_pool))
        for x in (h * G, h * G + G - 1):
            want, ls, A, big = O.attention(q[rows, x].double(), k, v, 128 ** -0.5, T - m + rows + 1)
            d = 2.0 ** -17 * big[:, None]
            p_round = 2.0 ** -8 if kv == "bf16" else 2.0 ** -11
            tol = (2.0 ** -8 + 2.0 ** -9) * want.abs() + (p_round + 2.0 ** -8 + 2 * d + 2.0 ** -18) * A
            assert bool((out[rows, x].double() - want).abs().le(tol).all()), (h, x)
            assert bool((lse[rows, x].double() - ls).abs().le(d[:, 0] + 2.0 ** -9 + 2.0 ** -23 * ls.abs()).all()), (h, x)
