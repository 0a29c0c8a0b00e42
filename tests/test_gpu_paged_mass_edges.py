"""Attention mass and eviction over the paged cache where they are easily wrong, on the GPU through the C ABI, against the
64-bit oracle.  Tolerances as in tests/test_gpu_paged_mass.py."""
import math

import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K
from compressed_kv_cache_vector_gb300.build import build
from tests.test_gpu_paged import Made, _gen, _i32
from tests.test_gpu_paged_mass import SCALE, _check_mass, _evict_check, _made_mass

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


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("news,G", [([20, 5, 1, 9, 3], 4), ([300, 70, 600, 9, 2], 4)])
@pytest.mark.parametrize("first", [256, 300, 511, 512, 4000, 10 ** 6])
def test_mass_from_a_token_behind_whole_tiles(kv, news, G, first):
    """Keys before `first` are left out of the work; sequences that end before it, at it and behind it."""
    lens = [6000, 500, 700, 257, 256]
    made = Made(kv, 32, 2, G, lens, 3, spread=3)
    cu = _cu(news)
    q = torch.randn(cu[-1], 2 * G, 128, generator=_gen(2), device=DEV).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table, _i32(cu), max(news), cu[-1])
    _, lse = made.c.prefill_attn(0, b, q, lse=True)
    for causal, add in ((True, True), (False, False)):
        if not causal:
            _, lse = made.c.prefill_attn(0, b, q, causal=False, lse=True)
        m = _made_mass(made, 2)
        before = m.mass.clone()
        made.c.prefill_mass(0, b, q, lse, m, causal=causal, first=first, add=add)
        assert made.c.poll_error() == (0, 0)
        _check_mass(made, before, m.mass, q, cu, news, SCALE, causal, add, first, lse)
    one = _made_mass(made, 4)
    before = one.mass.clone()
    step = K.PagedBatch(made.kv_len, made.table)
    made.c.decode_attn_mass(0, step, q[:5].contiguous(), one, first=first)
    assert made.c.poll_error() == (0, 0)
    _check_mass(made, before, one.mass, q, list(range(5)), [1] * 5, SCALE, True, True, first)


@pytest.mark.parametrize("kv,P,shared", [("bf16", 16, 528), ("e4m3", 64, 576), ("e4m3", 16, 256)])
@pytest.mark.parametrize("beyond", [0, 5, 200])
def test_sequences_that_share_pages_before_first(kv, P, shared, beyond):
    """Their logits for shared tokens meet in the same places and are no one's; the mass before `first` stays, to the
    bit, with `first` where the shared pages end, in a page of their own, and far behind."""
    lens = [900, 1400, shared + 1, 2000, 777]
    made = Made(kv, P, 2, 4, lens, 11, spread=2)
    for row in made.rows[1:]:
        row[:shared // P] = made.rows[0][:shared // P]
    made.table.copy_(_i32(made.rows))
    first = shared + beyond
    q = torch.randn(5, 8, 128, generator=_gen(2), device=DEV).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table)
    m = _made_mass(made, 2)
    before = m.mass.clone()
    out, lse = made.c.decode_attn_mass(0, b, q, m, first=first, lse=True)
    assert made.c.poll_error() == (0, 0)
    _check_mass(made, before, m.mass, q, list(range(5)), [1] * 5, SCALE, True, True, first)
    ref, ref_lse = made.c.decode_attn(0, b, q, lse=True)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    for news in ([30, 7, 1, 64, 3], [300, 70, 1, 400, 9]):                              # windows and prompts
        cu = _cu(news)
        q = torch.randn(cu[-1], 8, 128, generator=_gen(4), device=DEV).to(torch.bfloat16)
        b = K.PagedBatch(made.kv_len, made.table, _i32(cu), max(news), cu[-1])
        _, lse = made.c.prefill_attn(0, b, q, lse=True)
        for add in (True, False):
            before = m.mass.clone()
            made.c.prefill_mass(0, b, q, lse, m, first=first, add=add)
            assert made.c.poll_error() == (0, 0)
            _check_mass(made, before, m.mass, q, cu, news, SCALE, True, add, first, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_mass_through_prompt_eviction_and_steps(kv):
    """A prompt's mass in both layers, the eviction that moves it, then steps, eager and replayed from a graph: what each
    call adds, against the oracle over what the pages hold at that time; the new token's mass is set."""
    n, L, P, H, G, T = 2, 2, 16, 2, 4, 230
    c = K.PagedKV(K.make_paged_config(H * G, H, L, P, 64, n, K.MK_KV_E4M3 if kv == "e4m3" else K.MK_KV_BF16), DEV)
    table = torch.arange(n * 20, dtype=torch.int32, device=DEV).view(n, 20)
    g = _gen(12)
    mass = K.PagedMass(c)
    mass.mass.fill_(7.0)                                                                # whatever was there before
    lens, rows = _i32([T, T - 30]), 2 * T - 30

    def now(lengths, layer):
        made = Made.__new__(Made)
        made.kv, made.P, made.n_kv, made.G, made.lens, made.layer = kv, P, H, G, lengths, layer
        made.c, made.rows, made.table = c, table.tolist(), table
        return made

    cu = [0, T, rows]
    batch = K.PagedBatch(lens, table, _i32(cu), T, rows)
    keep, new_len = _i32([100, 90]), _i32([0, 0])
    kept = torch.zeros(L, n, H, 100, dtype=torch.int32, device=DEV)
    for l in range(L):
        k, v = (torch.randn(rows, H, 128, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
        q = torch.randn(rows, H * G, 128, generator=g, device=DEV).to(torch.bfloat16)
        c.append(l, batch, k, v)
        _, lse = c.prefill_attn(l, batch, q, lse=True)
        before = mass.mass.clone()
        c.prefill_mass(l, batch, q, lse, mass, add=False)
        made = now([T, T - 30], l)
        _check_mass(made, before, mass.mass, q, cu, [T, T - 30], SCALE, True, False, 0, lse)
        pools = {x: getattr(c, x + "_pool").view(torch.uint8).clone() for x in ("k", "v")}
        if kv == "e4m3":
            pools.update({x + "s": getattr(c, x + "_scale").clone() for x in ("k", "v")})
        before = mass.mass.clone()
        c.evict(l, batch, mass, keep, first=4, recent=20, kept=kept[l], new_len=new_len)
        assert c.poll_error() == (0, 0)
        _evict_check(made, pools, before, mass.mass, [100, 90], 4, 20, kept[l], new_len)
    step = K.PagedBatch(new_len, table)
    ks, vs = (torch.randn(L, n, H, 128, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    qs = torch.randn(L, n, H * G, 128, generator=g, device=DEV).to(torch.bfloat16)
    out = torch.zeros(L, n, H * G, 128, dtype=torch.bfloat16, device=DEV)

    def one():
        new_len.add_(1)
        for l in range(L):
            c.append(l, step, ks[l], vs[l])
            c.decode_attn_mass(l, step, qs[l], mass, out=out[l], first=4)

    def checked(call, count):
        before = mass.mass.clone()
        qs.copy_(torch.randn(qs.shape, generator=g, device=DEV))
        call()
        torch.cuda.synchronize()
        assert c.poll_error() == (0, 0) and new_len.tolist() == [100 + count, 90 + count]
        for l in range(L):
            was, is_now = before.clone(), mass.mass.clone()
            was[1 - l], is_now[1 - l] = 0, 0                                            # this layer's, the other's checked by itself
            _check_mass(now(new_len.tolist(), l), was, is_now, qs[l], [0, 1], [1, 1], SCALE, True, True, 4)

    checked(one, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    for i in range(2, 5):
        checked(graph.replay, i)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_calls_behind_an_error_leave_mass_and_rows(kv):
    """Steps, windows, prompts and shared prefixes do nothing until the error is cleared, and then what they should."""
    made = Made(kv, 16, 2, 4, [700, 300], 5)
    c, m = made.c, _made_mass(made, 2)
    q = torch.randn(400, 8, 128, generator=_gen(3), device=DEV).to(torch.bfloat16)
    step, cu = K.PagedBatch(made.kv_len, made.table), [0, 300, 400]
    few, many = (K.PagedBatch(made.kv_len, made.table, _i32(x), 300 if x[1] == 300 else 20, x[2]) for x in ([0, 20, 30], cu))
    lse = c.prefill_attn(0, many, q, lse=True)[1]
    few_lse = c.prefill_attn(0, few, q[:30], lse=True)[1]
    out, ls = torch.full((2, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV), torch.full((2, 8), 3.0, device=DEV)
    prefix = K.PagedPrefix(_i32([0, 2]), _i32([0]))
    before = m.mass.clone()
    c.evict(0, step, m, _i32([5, 5]), first=4, recent=4)                                # below what always stays: an error
    for call in (lambda: c.decode_attn_mass(0, step, q[:2], m, out=out, lse=ls), lambda: c.prefill_mass(0, few, q[:30], few_lse, m),
                 lambda: c.prefill_mass(0, many, q, lse, m), lambda: c.prefix_attn(0, step, prefix, q[:2], out=out, lse=ls)):
        call()
        assert c.poll_error() == (5, 16) and torch.equal(m.mass, before)
        assert bool((out == 3).all()) and bool((ls == 3).all())
    c.clear_error()
    c.prefill_mass(0, many, q, lse, m)
    assert c.poll_error() == (0, 0)
    _check_mass(made, before, m.mass, q, cu, [300, 100], SCALE, True, True, 0, lse)
