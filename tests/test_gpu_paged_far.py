"""Attention over the paged cache with queries whose channels, and keys whose scales, lie far apart, on the GPU through
the C ABI, against the 64-bit oracle.  Tolerances as in tests/test_gpu_paged.py."""
import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K
from compressed_kv_cache_vector_gb300.build import build
from tests.test_gpu_paged import Made, _check_attention, _gen, _i32

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _calls(made, q, scale, lens, P):
    """The calls that give single tokens' attention: (name, out, lse)."""
    c, b = made.c, K.PagedBatch(made.kv_len, made.table)
    n = len(lens)
    yield ("decode", *c.decode_attn(0, b, q, scale=scale, lse=True))
    yield ("mass", *c.decode_attn_mass(0, b, q, K.PagedMass(c), scale=scale, lse=True))
    yield ("prefix", *c.prefix_attn(0, b, K.PagedPrefix(_i32([0, n]), _i32([P])), q, scale=scale, lse=True))
    cu = _i32(list(range(n + 1)))
    yield ("several", *c.prefill_attn(0, K.PagedBatch(made.kv_len, made.table, cu, 2, n), q, scale=scale, lse=True))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("small", [0.0101, 2.0 ** -13])
def test_queries_with_one_channel_far_above_the_others(kv, small):
    """A channel of 1000 beside far smaller ones, in which no key has anything: the others alone make the logits."""
    lens = [950, 901, 33, 1200, 5000]
    made = Made(kv, 32, 2, 4, lens, 8)
    for row in made.rows[1:]:
        row[0] = made.rows[0][0]                                                        # for the prefix
    made.table.copy_(_i32(made.rows))
    made.c.k_pool[..., 5] = 0
    if kv == "e4m3":
        made.c.k_scale.mul_(1 / small)
    else:
        made.c.k_pool.mul_(1 / small)
    q = small * torch.randn(5, 8, 128, generator=_gen(2), device=DEV)
    q[..., 5] = 1000.0
    q = q.to(torch.bfloat16)
    for name, out, lse in _calls(made, q, SCALE, lens, 32):
        assert made.c.poll_error() == (0, 0), name
        _check_attention(made, q, out, lse, SCALE, [1] * 5, True, 2.0 ** -11)
    news, cu = [20, 64, 3, 40, 9], _i32([0, 20, 84, 87, 127, 136])                      # row tiles
    q = small * torch.randn(136, 8, 128, generator=_gen(3), device=DEV)
    q[..., 5] = 1000.0
    q = q.to(torch.bfloat16)
    out, lse = made.c.prefill_attn(0, K.PagedBatch(made.kv_len, made.table, cu, 64, 136), q, lse=True)
    assert made.c.poll_error() == (0, 0)
    _check_attention(made, q, out, lse, SCALE, news, True, 2.0 ** -8 if kv == "bf16" else 2.0 ** -11)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("up", [23, 25, 27, 29, 31, 40, 60])
@pytest.mark.parametrize("sign", [1, -1])
def test_logits_too_large_for_a_shift(kv, up, sign):
    """Keys of 2^up: next to the maximum a shift of its own size is lost in rounding.  Where one token is above the others
    by more than the logits' error, its value is the result, and its logit the sum's logarithm."""
    lens = [950, 901, 33, 1200, 5000]
    made = Made(kv, 16, 2, 4, lens, 8)
    for row in made.rows[1:]:
        row[0] = made.rows[0][0]                                                        # for the prefix
    made.table.copy_(_i32(made.rows))
    if kv == "e4m3":
        made.c.k_scale.mul_(2.0 ** up)
    else:
        made.c.k_pool.mul_(2.0 ** up)
    q = torch.randn(5, 8, 128, generator=_gen(2), device=DEV).to(torch.bfloat16)
    scale, seen = sign * SCALE, 0
    for name, out, lse in _calls(made, q, scale, lens, 16):
        assert made.c.poll_error() == (0, 0), name
        assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all()), name
        for i in range(5):
            for h in range(8):
                k, v = made.held(i, h // 4)
                z = k @ q[i, h].double() * scale
                d = 2.0 ** -17 * float((k.abs() @ q[i, h].double().abs()).max()) * abs(scale)
                two = torch.topk(z, 2)
                if float(two.values[0] - two.values[1]) < 4 * d + 60:
                    continue
                seen += 1
                want = v[two.indices[0]]
                assert bool(((out[i, h].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -11 * want.abs()).all()), (name, i, h)
                assert abs(float(lse[i, h]) - float(two.values[0])) <= d + 2.0 ** -22 * abs(float(two.values[0])), (name, i, h)
    assert seen > 100
