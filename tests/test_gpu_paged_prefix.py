"""Attention of single tokens for sequences that share prefixes, on the GPU through the C ABI, against the 64-bit oracle.

Tolerances as in tests/test_gpu_paged.py (fixed before the first run), with the weights' rounding of the shared tokens:
2^-11 (fp16, e4m3 cache) or 2^-8 (bf16 cache) of each.
"""
import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K
from compressed_kv_cache_vector_gb300.build import build
from tests.test_gpu_paged import Made, _check_attention, _gen, _i32

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROUND = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _shared(kv, P, n_kv, G, groups, seed, wide=True, **kw):
    """A cache whose groups share pages.  groups: [(tokens that name the same pages, [lengths of the sequences])].
    wide: a page table so wide that the call cannot know that its batch is small (96 MB at most, where every sequence
    reads what it shares by itself)."""
    lens = [t for _, ts in groups for t in ts]
    cols = (96 << 20) // (len(lens) * P * n_kv * 256) + 1 if wide else 2
    made = Made(kv, P, n_kv, G, lens, seed, extra_cols=cols, **kw)
    at, cu = 0, [0]
    for n, ts in groups:
        longest = at + max(range(len(ts)), key=lambda i: ts[i]) if ts else at
        for i in range(at, at + len(ts)):
            k = min(n, lens[i]) // P
            made.rows[i][:k] = made.rows[longest][:k]
        at += len(ts)
        cu.append(at)
    made.table.copy_(_i32(made.rows))
    return made, K.PagedPrefix(_i32(cu), _i32([n for n, _ in groups]))


def _run(made, prefix, scale=128 ** -0.5, seed=1, size=1.5, check=True):
    n, heads = len(made.lens), made.n_kv * made.G
    q = (size * torch.randn(n, heads, 128, generator=_gen(seed), device=DEV)).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table)
    out, lse = made.c.prefix_attn(made.layer, b, prefix, q, scale=scale, lse=True)
    assert made.c.poll_error() == (0, 0)
    if check:
        _check_attention(made, q, out, lse, scale, [1] * n, True, ROUND[made.kv])
    out2, lse2 = made.c.prefix_attn(made.layer, b, prefix, q, scale=scale, lse=True)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16)) and torch.equal(lse, lse2)
    return q, out, lse


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("P,n_kv,G,wide", [(16, 2, 4, True), (32, 1, 8, True), (64, 3, 1, True), (16, 1, 2, True), (32, 2, 4, False)])
def test_groups_of_every_shape(kv, P, n_kv, G, wide):
    """Prefixes within a page, of whole pages, beyond a sequence's length; sequences that end with the prefix, that hold
    nothing; groups of one and of none."""
    groups = [(300, [330, 301, 300, 700, 304]), (0, [40]), (128, [128, 128, 129]), (5, [20, 9]), (64, []), (200, [210]),
              (1000, [64, 0, 640, 90]), (259, [260 + 7 * i for i in range(20)])]
    made, prefix = _shared(kv, P, n_kv, G, groups, 40 + P, wide, spread=5)
    _run(made, prefix, 0.1)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,G,tokens", [(2, 1, 6000), (3, 4, 20000), (8, 4, 5000), (16, 4, 3000), (17, 4, 2500), (32, 4, 4100),
                                        (33, 4, 1300), (100, 4, 2000), (130, 1, 2000), (40, 8, 1500), (256, 2, 600)])
def test_rows_of_every_number(kv, n, G, tokens):
    made, prefix = _shared(kv, 32, 2, G, [(tokens, [tokens + 1 + 13 * (i % 9) for i in range(n)])], n, n_pages=None)
    _run(made, prefix)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_many_groups_of_long_prefixes(kv):
    """Cells in several runs, runs with several cells, a second layer."""
    groups = [(500 + 333 * i, [520 + 333 * i + 50 * j for j in range(2 + i % 5)]) for i in range(12)]
    made, prefix = _shared(kv, 16, 2, 4, groups, 3, n_layers=2, layer=1)
    _run(made, prefix)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_more_cells_than_runs(kv):
    """Many short shared prefixes and many kv heads: a run holds the end of a cell, whole ones and a beginning."""
    groups = [(150 + 97 * (i % 11), [160 + 97 * (i % 11) + 20 * j for j in range(2 + i % 3)]) for i in range(40)]
    made, prefix = _shared(kv, 32, 16, 1, groups, 3)
    _run(made, prefix)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [-0.1, 0.0, 3.0])
def test_scales_and_growing_logits(kv, scale):
    """Logits that pass their rows' bounds again and again, of several hundred, all equal, of the other sign."""
    made, prefix = _shared(kv, 32, 2, 4, [(3000, [3000 + 40 * i for i in range(7)])], 8)
    ids = torch.tensor(made.rows[0][:93], dtype=torch.long, device=DEV)
    if kv == "e4m3":
        made.c.k_scale[0, ids] *= torch.exp2(torch.arange(93, device=DEV).float() // 16)[:, None]
    else:
        made.c.k_pool[0, ids] = (made.c.k_pool[0, ids].float() * (1 + 0.1 * torch.arange(93, device=DEV)[:, None, None, None])).to(torch.bfloat16)
    _run(made, prefix, scale)


def test_v_scales_far_apart():
    made, prefix = _shared("e4m3", 16, 2, 4, [(900, [950, 900, 1200])], 8, spread=30)
    _run(made, prefix)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_one_shared_token_with_nearly_all_weight(kv):
    made, prefix = _shared(kv, 16, 1, 4, [(30000, [30001 + i for i in range(5)])], 8)
    c, row = made.c, made.rows[0]
    if kv == "e4m3":
        c.k_scale[0, row[0]] = 0.125
    c.k_pool[0, row[0], 0, 0] = 0
    c.k_pool[0, row[0], 0, 0, 0] = torch.tensor(64.0 if kv == "e4m3" else 8.0, device=DEV).to(c.k_pool.dtype)
    q = torch.zeros(5, 4, 128, device=DEV)
    q[:, :, 0] = torch.tensor([8.0, 16.0, 1.0, 600.0, 12.0], device=DEV)[:, None]
    q = q.to(torch.bfloat16)
    out, lse = c.prefix_attn(0, K.PagedBatch(made.kv_len, made.table), prefix, q, lse=True)
    assert c.poll_error() == (0, 0)
    _check_attention(made, q, out, lse, 128 ** -0.5, [1] * 5, True, ROUND[kv])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_rows_strided_padded_absent_and_on_a_stream(kv):
    """Padded rows stay as they were; sequences without a token in the call, or padded ones without keys, do not stop the
    others from sharing and are given nothing, or zeros."""
    made, prefix = _shared(kv, 16, 2, 2, [(200, [230, 260, 0, 210, 333, 201])], 6)
    made.rows[2] = [-7] * len(made.rows[2])
    wide = torch.randn(10, 10 * 128, generator=_gen(5), device=DEV).to(torch.bfloat16)
    q = wide[:, 128:128 * 5].view(10, 4, 128)
    res = torch.full((10, 6, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((10, 4), 5.0, device=DEV)
    b = K.PagedBatch(made.kv_len, made.table, _i32([1, 2, 3, 4, 4, 5, 6]), 1, 10)       # the fourth has no token
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    made.c.prefix_attn(0, b, prefix, q, out=res[:, 1:5], lse=lse, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert made.c.poll_error() == (0, 0)
    _check_attention(made, q, res[:, 1:5], lse, 128 ** -0.5, [1, 1, 1, 0, 1, 1], True, ROUND[kv], starts=[1, 2, 3, 4, 4, 5])
    assert not bool(res[3, 1:5].any()) and bool(torch.isinf(lse[3]).all())
    assert bool((res[0] == 3).all()) and bool((res[6:] == 3).all()) and bool((res[:, 0] == 3).all()) and bool((res[:, 5] == 3).all())
    assert bool((lse[0] == 5).all()) and bool((lse[6:] == 5).all())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_captured_with_groups_that_change(kv):
    groups = [(640, [700, 650, 800, 900]), (320, [400, 500, 330])]
    made, prefix = _shared(kv, 32, 2, 4, groups, 4)
    q = torch.randn(7, 8, 128, generator=_gen(2), device=DEV).to(torch.bfloat16)
    out, lse = torch.zeros_like(q), torch.zeros(7, 8, device=DEV)
    b = K.PagedBatch(made.kv_len, made.table)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made.c.prefix_attn(0, b, prefix, q, out=out, lse=lse)
    for cu, shared in (([0, 4, 7], [640, 320]), ([0, 2, 4], [100, 31]), ([1, 1, 4], [640, 640]), ([0, 4, 7], [0, 320])):
        prefix.cu_group.copy_(_i32(cu))
        prefix.prefix_len.copy_(_i32(shared))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert made.c.poll_error() == (0, 0)
        _check_attention(made, q, out, lse, 128 ** -0.5, [1] * 7, True, ROUND[kv])


@pytest.mark.parametrize("wide", [True, False])
def test_wrong_groups_share_nothing_and_are_told(wide):
    made, prefix = _shared("bf16", 16, 2, 2, [(160, [200, 300, 170]), (64, [100, 90])], 6, wide)
    q = torch.randn(5, 4, 128, generator=_gen(2), device=DEV).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table)
    for cu, shared in (([0, 4, 3], [160, 64]), ([0, 3, 6], [160, 64]), ([-1, 3, 5], [160, 64]), ([0, 3, 5], [160, -1])):
        out, lse = made.c.prefix_attn(0, b, K.PagedPrefix(_i32(cu), _i32(shared)), q, lse=True)
        assert made.c.poll_error() == (5, 16)
        made.c.clear_error()
        _check_attention(made, q, out, lse, 128 ** -0.5, [1] * 5, True, ROUND["bf16"])
    # no groups at all: plain decode attention
    none = K.PagedPrefix(_i32([0]), _i32([]))
    assert torch.equal(made.c.prefix_attn(0, b, none, q), made.c.decode_attn(0, b, q))
    # a shared page id that is none
    made.table[0, 2] = 10 ** 6
    made.c.prefix_attn(0, b, prefix, q)
    assert made.c.poll_error() == (5, 17)
    made.c.clear_error()


def test_a_nan_key_reaches_the_rows_that_see_it():
    """A NaN among the shared keys reaches its group and no other; one among a sequence's own keys that sequence alone."""
    made, prefix = _shared("bf16", 16, 1, 4, [(640, [700, 650, 800]), (320, [400, 500, 330])], 4)
    made.c.k_pool[0, made.rows[0][5], 0, 3] = float("nan")
    made.c.k_pool[0, made.rows[4][22], 0, 3] = float("nan")                            # token 355 of the fifth
    q = torch.randn(6, 4, 128, generator=_gen(2), device=DEV).to(torch.bfloat16)
    out, lse = made.c.prefix_attn(0, K.PagedBatch(made.kv_len, made.table), prefix, q, lse=True)
    bad = torch.isnan(out.float()).flatten(1).all(dim=1)
    assert bad.tolist() == [True, True, True, False, True, False] and torch.isnan(lse).all(dim=1).tolist() == bad.tolist()
    assert not bool(torch.isnan(out[[3, 5]].float()).any())
