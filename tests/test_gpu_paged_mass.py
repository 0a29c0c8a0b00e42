"""Attention mass and eviction over the paged cache on the GPU, through the C ABI, against the 64-bit oracle.

Tolerances (fixed before the first run).  A weight w = exp(z - lse): the logit's fp32 sum of 128 products is off by at
most d = 128 * 2^-24 * sum |q k| scale; its product with the scale factors and the difference in base 2 by 3 roundings of
2^-24 (|z| + |lse|) log2 e < 2^-21 (|z| + |lse|); where the kernel forms the row's sum itself (a decode step), lse by
d + 2^-18 more; the exponential by 2^-21.  So w (2^-16 big + 2^-17), with big = largest sum |q k| scale of the row plus
|lse|.  Sums of n weights in 32 bits: n 2^-24 of the total, and as much of the mass held before.
"""
import ctypes
import math

import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K
from compressed_kv_cache_vector_gb300.build import build
from oracle import paged_oracle as O
from tests.test_gpu_paged import Made, _check_attention, _gen, _i32

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _made_mass(made, seed):
    m = K.PagedMass(made.c)
    m.mass.copy_(torch.rand(m.mass.shape, generator=_gen(seed), device=DEV))
    return m


def _of(made, mass, i, h):
    """The mass of one sequence's tokens and head, as doubles."""
    ids = torch.tensor(made.rows[i][: -(-made.lens[i] // made.P)], dtype=torch.long, device=DEV)
    return mass[made.layer, ids, h].double().reshape(-1)[: made.lens[i]]


def _check_mass(made, before, after, q, starts, news, scale, causal, add, first=0, lse=None):
    touched = torch.zeros_like(before, dtype=torch.bool)
    for i, (t, m) in enumerate(zip(made.lens, news)):
        if m == 0:
            continue
        see = torch.arange(m, device=DEV) + t - m + 1 if causal else torch.full((m,), t, device=DEV)
        j = torch.arange(min(first, t), t, device=DEV)
        touched[made.layer, torch.tensor(made.rows[i], device=DEV)[j // made.P], :, j % made.P] = True
        for h in range(made.n_kv):
            k, _ = made.held(i, h)
            want = torch.zeros(t, dtype=torch.float64, device=DEV)
            tol = torch.zeros_like(want)
            for g in range(made.G):
                rows = slice(starts[i], starts[i] + m)
                ls = None if lse is None else lse[rows, h * made.G + g].double()
                w, big = O.mass(q[rows, h * made.G + g].double(), k, scale, see.clamp(min=0), ls)
                want += w
                tol += 2.0 ** -16 * big + 2.0 ** -17 * w
            old = _of(made, before, i, h).clone()
            if not add:
                old[:] = 0
            elif causal:
                old[max(0, t - m):] = 0
            tol += (want + old) * (m * made.G + 2) * 2.0 ** -24 + 1e-37
            got = _of(made, after, i, h)[first:]
            err = (got - (want + old)[first:]).abs()
            assert bool(err.le(tol[first:]).all()), (i, h, float((err / tol[first:]).max()))
    assert torch.equal(before[~touched], after[~touched])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("P,n_kv,G", [(16, 2, 4), (32, 1, 8), (64, 3, 1), (16, 1, 2)])
def test_decode_step_leaves_mass(kv, P, n_kv, G):
    lens = [1, 40, 0, 129, 31, 64, 333, 12, 17, 2000]
    made = Made(kv, P, n_kv, G, lens, 5 + P, spread=4)
    q = (1.5 * torch.randn(len(lens), n_kv * G, 128, generator=_gen(1), device=DEV)).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table)
    ref, ref_lse = made.c.decode_attn(0, b, q, scale=0.1, lse=True)
    for first in (0, 37):
        m = _made_mass(made, 2)
        before = m.mass.clone()
        out, lse = made.c.decode_attn_mass(0, b, q, m, first=first, scale=0.1, lse=True)
        assert made.c.poll_error() == (0, 0)
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
        _check_mass(made, before, m.mass, q, list(range(len(lens))), [1] * len(lens), 0.1, True, True, first)


@pytest.mark.parametrize("kv,lens,G", [("e4m3", [70000], 4), ("bf16", [30000, 1, 9000], 8), ("e4m3", [5000] * 40, 2)])
def test_decode_step_mass_of_long_sequences(kv, lens, G):
    """Units in several CTAs' runs; rows of a second layer."""
    made = Made(kv, 64, 2, G, lens, 9, n_layers=2, layer=1)
    q = torch.randn(len(lens), 2 * G, 128, generator=_gen(2), device=DEV).to(torch.bfloat16)
    m = _made_mass(made, 3)
    before = m.mass.clone()
    b = K.PagedBatch(made.kv_len, made.table)
    out = made.c.decode_attn_mass(1, b, q, m)
    assert made.c.poll_error() == (0, 0)
    assert torch.equal(out, made.c.decode_attn(1, b, q))
    _check_mass(made, before, m.mass, q, list(range(len(lens))), [1] * len(lens), SCALE, True, True)
    assert torch.equal(before[0], m.mass[0])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("causal,add", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("P,n_kv,G", [(16, 2, 4), (32, 1, 8), (64, 3, 1), (16, 2, 2)])
def test_prompt_mass_ragged(kv, causal, add, P, n_kv, G):
    """Queries before and past tile borders, no new tokens, an empty context, more queries than keys, NaN behind every
    length, scales apart."""
    lens = [0, 1, 40, 129, 200, 64, 333, 12, 5, 700]
    news = [3, 1, 0, 129, 7, 64, 130, 33, 2, 257]
    made = Made(kv, P, n_kv, G, lens, 50 + P + G, spread=6)
    cu = [0]
    for x in news:
        cu.append(cu[-1] + x)
    rows = cu[-1]
    q = (1.5 * torch.randn(rows + 2, n_kv * G, 128, generator=_gen(G), device=DEV)).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table, _i32(cu), max(news), rows + 2)
    _, lse = made.c.prefill_attn(0, b, q, causal=causal, scale=0.11, lse=True)
    first = 0 if add else 21
    m = _made_mass(made, 4)
    before = m.mass.clone()
    made.c.prefill_mass(0, b, q, lse, m, causal=causal, first=first, add=add, scale=0.11)
    assert made.c.poll_error() == (0, 0)
    _check_mass(made, before, m.mass, q, cu, news, 0.11, causal, add, first, lse)
    again = K.PagedMass(made.c, before.clone())
    made.c.prefill_mass(0, b, q, lse, again, causal=causal, first=first, add=add, scale=0.11)
    assert torch.equal(again.mass, m.mass)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("news,lens,G,scale", [([600], [600], 4, SCALE), ([513], [4100], 4, -SCALE), ([2, 4], [6000, 3333], 4, 0.2),
                                               ([300], [1500], 1, SCALE), ([9], [20000], 8, 0.0),
                                               ([40, 900, 33, 500, 3, 1200], [3000, 2500, 4000, 700, 2600, 1200], 4, SCALE)])
def test_prompt_mass_longer(kv, news, lens, G, scale):
    made = Made(kv, 32, 2, G, lens, 7)
    cu = [0]
    for x in news:
        cu.append(cu[-1] + x)
    wide = torch.randn(cu[-1], (2 * G + 2) * 128, generator=_gen(3), device=DEV).to(torch.bfloat16)
    q = wide[:, 128:128 + 2 * G * 128].view(cu[-1], 2 * G, 128)                        # strided rows
    b = K.PagedBatch(made.kv_len, made.table, _i32(cu), max(news), cu[-1])
    _, lse = made.c.prefill_attn(0, b, q, scale=scale, lse=True)
    m = _made_mass(made, 5)
    before = m.mass.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    made.c.prefill_mass(0, b, q, lse, m, scale=scale, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert made.c.poll_error() == (0, 0)
    _check_mass(made, before, m.mass, q, cu, news, scale, True, True, 0, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("causal,add", [(True, False), (False, True)])
@pytest.mark.parametrize("P,n_kv,G,top", [(16, 2, 4, 64), (32, 3, 8, 32), (64, 1, 2, 64), (32, 16, 1, 100), (16, 2, 8, 16)])
def test_window_mass(kv, causal, add, P, n_kv, G, top):
    """Up to 256 rows a kv head: one row tile or two, keys that the first tile does not see, many sequences, long ones."""
    lens = [0, 1, 40, 129, 5000, 256, 333, 12, 5, 700, 257, 9000] + [100 + 31 * i for i in range(20)]
    news = [3, 1, 0, top, 7, 33, 16, 9, 2, top - 1, top // 2, 1] + [1 + i % 13 for i in range(20)]
    news = [min(x, top) for x in news]
    made = Made(kv, P, n_kv, G, lens, 50 + P + G, spread=6)
    cu = [0]
    for x in news:
        cu.append(cu[-1] + x)
    rows = cu[-1]
    wide = (1.5 * torch.randn(rows + 2, (n_kv * G + 1) * 128, generator=_gen(G), device=DEV)).to(torch.bfloat16)
    wide[rows:] = float("nan")                                                          # padding rows are no one's
    q = wide[:, :n_kv * G * 128].view(rows + 2, n_kv * G, 128)
    b = K.PagedBatch(made.kv_len, made.table, _i32(cu), top, rows + 2)
    _, lse = made.c.prefill_attn(0, b, q, causal=causal, scale=0.11, lse=True)
    m = _made_mass(made, 4)
    before = m.mass.clone()
    made.c.prefill_mass(0, b, q, lse, m, causal=causal, first=7, add=add, scale=0.11)
    assert made.c.poll_error() == (0, 0)
    _check_mass(made, before, m.mass, q, cu, news, 0.11, causal, add, 7, lse)
    again = K.PagedMass(made.c, before.clone())
    made.c.prefill_mass(0, b, q, lse, again, causal=causal, first=7, add=add, scale=0.11)
    assert torch.equal(again.mass, m.mass)


def test_mass_sums_to_the_queries_and_a_nan_key_is_alone():
    """Every query hands out a total weight of 1; a key of NaN has a mass of NaN and spoils no other's."""
    made = Made("bf16", 16, 2, 4, [700, 90], 3)
    cu, n = [0, 300, 390], 390
    q = torch.randn(n, 8, 128, generator=_gen(3), device=DEV).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table, _i32(cu), 300, n)
    _, lse = made.c.prefill_attn(0, b, q, lse=True)
    m = K.PagedMass(made.c)
    made.c.prefill_mass(0, b, q, lse, m, add=False)
    for i, x in enumerate((300, 90)):
        for h in range(2):
            assert abs(float(_of(made, m.mass, i, h).sum()) - 4 * x) < 1e-4 * 4 * x
    clean = m.mass.clone()
    made.c.k_pool[0, made.rows[0][3], 1, 5] = float("nan")                              # token 53 of the first sequence
    made.c.prefill_mass(0, b, q, lse, m, add=False)
    w = _of(made, m.mass, 0, 1)
    assert math.isnan(float(w[53])) and int(torch.isnan(m.mass).sum()) == 1
    keep = torch.ones_like(m.mass, dtype=torch.bool)
    keep[0, made.rows[0][3], 1, 5] = False
    assert torch.equal(m.mass[keep], clean[keep])
    assert made.c.poll_error() == (0, 0)


# ---- eviction --------------------------------------------------------------------------------------------------------

def _evict_check(made, before, mass_before, mass, keeps, first, recent, kept, new_len):
    """kept, new_len, mass, codes and scales against the definition, and nothing else written."""
    c, P, lay = made.c, made.P, made.layer
    es = 1 if made.kv == "e4m3" else 2
    raw = {x: getattr(c, x + "_pool").view(torch.uint8) for x in ("k", "v")}
    free = torch.zeros(c.cfg.n_pages, made.n_kv, P, dtype=torch.bool, device=DEV)       # slots that may hold anything
    fixed = torch.ones(c.cfg.n_pages, made.n_kv, dtype=torch.bool, device=DEV)
    for i, t in enumerate(made.lens):
        n = min(t, keeps[i])
        assert int(new_len[i]) == n
        for h in range(made.n_kv):
            w = _of(made, mass_before, i, h)
            stay = O.evict_tokens(w.tolist(), keeps[i], first, recent)
            assert kept[i, h, :n].tolist() == stay, (i, h)
            if n == t:
                continue
            src = torch.tensor(stay, dtype=torch.long, device=DEV)
            ids = torch.tensor(made.rows[i][: -(-t // P)], dtype=torch.long, device=DEV)
            for j in range(-(-t // P)):
                page, a, e = made.rows[i][j], j * P, min(n, (j + 1) * P)
                if a >= n or stay[e - 1] != e - 1:
                    free[page, h, max(0, n - a) if a < n else 0:] = True
                if a >= n:
                    continue
                if stay[e - 1] == e - 1:                                                # all stay: untouched
                    continue
                fixed[page, h] = False
                s = src[a:e]
                got = mass[lay, page, h, : e - a].double()
                want = w[s]
                assert torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)])
                for x in ("k", "v"):
                    pool = raw[x][lay].view(c.cfg.n_pages, made.n_kv, P, 128 * es)
                    old = before[x][lay].view(c.cfg.n_pages, made.n_kv, P, 128 * es)[ids[s // P], h, s % P]
                    new = pool[page, h, : e - a]
                    if es == 2:
                        assert torch.equal(old, new)
                        continue
                    y = old.view(torch.float8_e4m3fn).double() * before[x + "s"][lay, ids[s // P], h].double()[:, None]
                    y = y.float().double()
                    fine = y.abs()[torch.isfinite(y)]
                    one = O.scale_of(float(fine.max()) if fine.numel() else 0.0)
                    assert float(getattr(c, x + "_scale")[lay, page, h]) == one, (i, h, j)
                    code = O.e4m3_round(y / one)
                    got = new.view(torch.float8_e4m3fn).double()
                    assert torch.equal(torch.isnan(code), torch.isnan(got))
                    assert torch.equal(code[~torch.isnan(code)], got[~torch.isnan(code)]), (i, h, j)
                free[page, h, : e - a] = True                                           # checked
    for x in ("k", "v"):
        same = raw[x][lay].view(c.cfg.n_pages, made.n_kv, P, -1) == before[x][lay].view(c.cfg.n_pages, made.n_kv, P, -1)
        assert bool((same.all(dim=3) | free).all())
        if es == 1:
            s0, s1 = before[x + "s"][lay], getattr(c, x + "_scale")[lay]
            assert bool(((s0 == s1) | (torch.isnan(s0) & torch.isnan(s1)) | ~fixed).all())
    m0, m1 = mass_before[lay], mass[lay]
    assert bool(((m0 == m1) | (torch.isnan(m0) & torch.isnan(m1)) | free).all())


def _evict_run(made, keeps, first, recent, seed, tweak=None, **kw):
    c = made.c
    m = K.PagedMass(c)
    m.mass.copy_(torch.exp(2 * torch.randn(m.mass.shape, generator=_gen(seed), device=DEV)))
    m.mass[torch.rand(m.mass.shape, generator=_gen(seed + 1), device=DEV) < 0.1] = 0.0
    if tweak:
        tweak(m.mass)
    before = {x: getattr(c, x + "_pool").view(torch.uint8).clone() for x in ("k", "v")}
    if made.kv == "e4m3":
        before.update({x + "s": getattr(c, x + "_scale").clone() for x in ("k", "v")})
    was = m.mass.clone()
    new_len, kept = c.evict(made.layer, K.PagedBatch(made.kv_len, made.table), m, _i32(keeps), first=first, recent=recent, **kw)
    assert c.poll_error() == (0, 0)
    _evict_check(made, before, was, m.mass, keeps, first, recent, kept, new_len)
    return m, new_len, kept


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("P,n_kv", [(16, 2), (32, 1), (64, 3)])
@pytest.mark.parametrize("first,recent", [(0, 0), (4, 16), (70, 1)])
def test_evict_ragged(kv, P, n_kv, first, recent):
    lens = [0, 1, 200, 129, 64, 65, 333, 90, 128, 700]
    keeps = [0, 5, 100, 128, 64, 71, 332, 0 if first + recent == 0 else first + recent, 127, 300]
    made = Made(kv, P, n_kv, 2, lens, 20 + P, spread=5)
    _evict_run(made, keeps, first, recent, 3)


@pytest.mark.parametrize("kv,P", [("bf16", 16), ("e4m3", 64), ("e4m3", 16)])
@pytest.mark.parametrize("lens,keeps", [([70000], [17000]), ([9000, 30000, 500], [8990, 64, 200]), ([3000] * 30, [1500] * 30),
                                        ([120000, 64], [100000, 1])])
def test_evict_long(kv, P, lens, keeps):
    """Slices that outgrow shared memory, one to eight CTAs a head, many items that read each other's slots."""
    made = Made(kv, P, 2, 1, lens, 31, spread=3, n_layers=2, layer=1)
    _evict_run(made, keeps, 0, 0, 9)


def test_evict_ties_infinities_and_nan():
    made = Made("e4m3", 16, 2, 4, [500, 500, 500], 6)

    def tweak(w):
        w[:, made.rows[0][:40]] = 1.0                                                    # all equal: the lowest numbers
        w[:, made.rows[1][3]] = math.nan
        w[:, made.rows[1][4]] = math.inf
        w[:, made.rows[1][5]] = -math.inf
        w[:, made.rows[2][:40]] = -0.0
        w[:, made.rows[2][9]] = 0.0

    _evict_run(made, [100, 490, 250], 3, 5, 4, tweak)


def test_evict_large_values_move_into_fine_pages():
    """A page of tiny values gets a huge token from behind: its scale grows, small codes round; and the other way."""
    made = Made("e4m3", 16, 1, 1, [64], 2)
    made.c.k_scale[0, made.rows[0]] = torch.exp2(torch.tensor([-20., 3., -60., 40.] + [0.] * 2, device=DEV))[:, None]
    made.c.v_scale[0, made.rows[0]] = 0.37                                               # no power of two

    def tweak(w):
        flat = torch.zeros(64, device=DEV)
        flat[[0, 1, 17, 33, 34, 50]] = 5.0
        flat[[2, 18, 51]] = 4.0
        w[0, made.rows[0][:4], 0] = flat.view(4, 16)

    _evict_run(made, [9], 0, 0, 1, tweak)


@pytest.mark.parametrize("kv,P,first", [("bf16", 16, 80), ("e4m3", 16, 16), ("e4m3", 32, 100)])
def test_evict_behind_a_shared_prefix(kv, P, first):
    """Sequences whose first pages are the same, in the middle of 64 slots: each waits for its own readers alone."""
    lens = [12000 - 700 * i for i in range(14)]
    made = Made(kv, P, 2, 1, lens, 41, spread=2)
    for row in made.rows[1:]:
        row[:first // P] = made.rows[0][:first // P]
    made.table.copy_(_i32(made.rows))
    _evict_run(made, [t - 64 - 100 * i for i, t in enumerate(lens)], first, 7, 5)


def test_step_evict_step_and_captured():
    """A run of them as they are used: a prompt, its mass, eviction in both layers, then steps that append with positions
    of their own and count mass, eager and captured; against the oracle over what the pages hold."""
    n, L, P, H, G, T = 2, 2, 16, 2, 4, 230
    cfg = K.make_paged_config(H * G, H, L, P, 64, n, K.MK_KV_E4M3)
    c = K.PagedKV(cfg, DEV)
    table = torch.arange(n * 20, dtype=torch.int32, device=DEV).view(n, 20)
    rope_t = K.rope_table(512, 128)
    g = _gen(12)
    mass = K.PagedMass(c)
    lens = _i32([T, T - 30])
    cu, rows = _i32([0, T, 2 * T - 30]), 2 * T - 30
    batch = K.PagedBatch(lens, table, cu, T, rows)
    keep, new_len = _i32([100, 90]), _i32([0, 0])
    kept = torch.zeros(L, n, H, 100, dtype=torch.int32, device=DEV)
    for l in range(L):
        k, v = (torch.randn(rows, H, 128, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
        q = torch.randn(rows, H * G, 128, generator=g, device=DEV).to(torch.bfloat16)
        q = c.append(l, batch, k, v, rope=K.Rope(rope_t, 128), q=q)
        _, lse = c.prefill_attn(l, batch, q, lse=True)
        c.prefill_mass(l, batch, q, lse, mass, add=False)
        c.evict(l, batch, mass, keep, first=4, recent=20, kept=kept[l], new_len=new_len)
    assert c.poll_error() == (0, 0) and new_len.tolist() == [100, 90]
    assert kept[0, 0, 0, :4].tolist() == [0, 1, 2, 3] and kept[1, 1, 1, 70:90].tolist() == list(range(180, 200))
    # steps
    pos = _i32([T, T - 30])
    step = K.PagedBatch(new_len, table)
    rope = K.Rope(rope_t, 128, positions=pos)
    ks, vs = (torch.randn(L, n, H, 128, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    qs = torch.randn(L, n, H * G, 128, generator=g, device=DEV).to(torch.bfloat16)
    out = torch.zeros(L, n, H * G, 128, dtype=torch.bfloat16, device=DEV)
    qr = torch.zeros_like(qs)

    def one():
        new_len.add_(1)
        pos.add_(1)
        for l in range(L):
            c.append(l, step, ks[l], vs[l], rope=rope, q=qs[l], q_out=qr[l])
            c.decode_attn_mass(l, step, qr[l], mass, out=out[l], first=4)

    pos.sub_(1)
    one()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert c.poll_error() == (0, 0) and new_len.tolist() == [104, 94] and pos.tolist() == [T + 3, T - 27]

    class Now:
        pass

    for l in range(L):
        now = Made.__new__(Made)
        now.kv, now.P, now.n_kv, now.G, now.lens, now.layer = "e4m3", P, H, G, new_len.tolist(), l
        now.c, now.rows, now.table, now.kv_len = c, table.tolist(), table, new_len
        ref, lse = c.decode_attn(l, step, qr[l], lse=True)
        assert torch.equal(ref, out[l])
        _check_attention(now, qr[l], ref, lse, SCALE, [1, 1], True, 2.0 ** -11)


def test_evict_in_a_graph_replayed_with_new_lengths():
    made = Made("e4m3", 32, 2, 2, [900, 400], 5)
    c, m = made.c, K.PagedMass(made.c)
    m.mass.uniform_(generator=_gen(1))
    b = K.PagedBatch(made.kv_len, made.table)
    keep, new_len = _i32([300, 400]), _i32([0, 0])
    kept = torch.zeros(2, 2, 900, dtype=torch.int32, device=DEV)
    saved = [t.clone() for t in (c.k_pool.view(torch.uint8), c.v_pool.view(torch.uint8), c.k_scale, c.v_scale, m.mass)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.evict(0, b, m, keep, first=2, recent=8, kept=kept, new_len=new_len)
    for keeps in ([300, 400], [37, 50], [899, 10]):
        for t, s in zip((c.k_pool.view(torch.uint8), c.v_pool.view(torch.uint8), c.k_scale, c.v_scale, m.mass), saved):
            t.copy_(s)
        keep.copy_(_i32(keeps))
        graph.replay()
        torch.cuda.synchronize()
        assert c.poll_error() == (0, 0)
        _evict_check(made, {"k": saved[0], "v": saved[1], "ks": saved[2], "vs": saved[3]}, saved[4], m.mass, keeps, 2, 8, kept, new_len)


def test_device_errors_leave_other_sequences_right():
    """A keep below what always stays, one above the columns of kept, a length beyond the table, a page id that is none."""
    made = Made("bf16", 16, 2, 2, [100, 100, 100, 100, 100], 5, extra_cols=1)
    made.kv_len[2] = 16 * made.table.shape[1] + 1
    made.table[3, 2] = 999
    c, m = made.c, K.PagedMass(made.c)
    m.mass.uniform_(generator=_gen(1))
    was = m.mass.clone()
    before = c.k_pool.clone()
    kept = torch.full((5, 2, 50), -1, dtype=torch.int32, device=DEV)
    new_len, _ = c.evict(0, K.PagedBatch(made.kv_len, made.table), m, _i32([5, 51, 40, 40, 40]), first=4, recent=4, kept=kept)
    st, detail = c.poll_error()
    assert st == 5 and detail in (16, 17)
    assert new_len.tolist()[:3] == [100, 100, 16 * made.table.shape[1] + 1] and new_len.tolist()[4] == 40
    for i in (0, 1):
        ids = made.rows[i][:7]
        assert torch.equal(c.k_pool[0, ids].view(torch.int16), before[0, ids].view(torch.int16))
    for h in range(2):
        assert kept[4, h, :40].tolist() == O.evict_tokens(_of(made, was, 4, h).tolist(), 40, 4, 4)
    # the next call does nothing until the error is cleared
    again = torch.full_like(kept, -1)
    good = K.PagedBatch(_i32([100] * 5), torch.cat([made.table[4:5]] * 5))
    c.evict(0, good, m, _i32([100] * 5), kept=torch.full((5, 2, 100), -1, dtype=torch.int32, device=DEV))
    c.clear_error()
    assert bool((again == -1).all())


def test_eviction_waits_for_nobody_over_a_bad_page():
    """A page id that is none at the first of 64 slots: who reads there cannot be told, and is not waited for (a wait
    that runs out takes 200 ms)."""
    made = Made("e4m3", 16, 1, 1, [5000, 300], 5)
    for j in (128, 160):
        made.table[0, j] = 99999
    c, m = made.c, K.PagedMass(made.c)
    m.mass.uniform_(generator=_gen(1))
    was, b, keep = m.mass.clone(), K.PagedBatch(made.kv_len, made.table), _i32([4000, 200])
    c.evict(0, K.PagedBatch(_i32([0, 0]), made.table), m, keep)                           # loads the kernels
    a, e = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    a.record()
    new_len, kept = c.evict(0, b, m, keep, first=100, recent=4)
    e.record()
    e.synchronize()
    assert a.elapsed_time(e) < 100 and c.poll_error() == (5, 17)
    assert new_len.tolist() == [4000, 200] and kept[1, 0, :200].tolist() == O.evict_tokens(_of(made, was, 1, 0).tolist(), 200, 100, 4)


def test_a_bad_page_does_not_reach_other_sequences_mass():
    """A page id that is none is read as page 0, whose own sequence keeps its logits."""
    made = Made("e4m3", 16, 2, 4, [300, 200], 5)
    c = made.c
    zero = int((made.table[1] == 0).any())                                              # the sequence that owns page 0
    owner, other = (1, 0) if zero else (0, 1)
    if not bool((made.table[owner] == 0).any()):                                        # page 0 is free: give it to one
        j = 3
        old = made.rows[owner][j]
        for x in ("k", "v"):
            getattr(c, x + "_pool").view(torch.uint8)[0, 0] = getattr(c, x + "_pool").view(torch.uint8)[0, old]
            getattr(c, x + "_scale")[0, 0] = getattr(c, x + "_scale")[0, old]
        made.rows[owner][j] = 0
        made.table[owner, j] = 0
    made.table[other, 5] = 12345
    q = torch.randn(2, 8, 128, generator=_gen(1), device=DEV).to(torch.bfloat16)
    m = _made_mass(made, 2)
    before = m.mass.clone()
    c.decode_attn_mass(0, K.PagedBatch(made.kv_len, made.table), q, m)
    assert c.poll_error() == (5, 17)
    for h in range(2):
        k, _ = made.held(owner, h)
        w = sum(O.mass(q[owner:owner + 1, h * 4 + g].double(), k, SCALE, torch.full((1,), made.lens[owner], device=DEV))[0] for g in range(4))
        old = _of(made, before, owner, h).clone()
        old[-1] = 0
        assert float((_of(made, m.mass, owner, h) - old - w).abs().max()) < 1e-4


def test_refusals():
    """Every argument that a call can check before it launches anything."""
    made = Made("e4m3", 16, 2, 4, [40, 40], 5)
    c, b = made.c, K.PagedBatch(made.kv_len, made.table)
    m = K.PagedMass(c)
    lib, ref, g = c.lib, b.ref, 1 << 20
    two = K.PagedBatch(made.kv_len, made.table, _i32([0, 2, 4]), 2, 4)

    def dec(batch=ref, q=g, scale=0.1, out=g, mass=g, first=0, scratch=g, size=1 << 40, layer=0):
        return lib.mk_paged_decode_attn_mass(c.h, layer, batch, q, 1024, scale, out, 1024, None, mass, first, scratch, size, None)

    assert dec(batch=two.ref) == 1 and dec(q=g + 2) == 1 and dec(mass=0) == 1 and dec(mass=g + 2) == 1 and dec(first=-1) == 1
    assert dec(scratch=0) == 1 and dec(scratch=g + 8) == 1 and dec(size=m.scratch_bytes - 1) == 2 and dec(layer=1) == 1
    assert dec(scale=math.inf) == 1

    def pre(q=g, lse=g, mass=g, first=0, add=1, causal=1, scale=0.1, stride=1024):
        return lib.mk_paged_prefill_mass(c.h, 0, two.ref, causal, q, stride, scale, lse, mass, first, add, None)

    assert pre(q=0) == 1 and pre(lse=0) == 1 and pre(lse=g + 1) == 1 and pre(mass=0) == 1 and pre(first=-1) == 1 and pre(add=2) == 1
    assert pre(causal=2) == 1 and pre(scale=math.nan) == 1 and pre(stride=1020) == 1

    def ev(mass=g, keep=g, first=0, recent=0, kept=g, stride=8, new=g, batch=ref):
        return lib.mk_paged_evict(c.h, 0, batch, mass, keep, first, recent, kept, stride, new, None)

    assert ev(mass=0) == 1 and ev(keep=0) == 1 and ev(first=-1) == 1 and ev(recent=-1) == 1 and ev(kept=0) == 1 and ev(stride=-1) == 1
    assert ev(new=0) == 1 and ev(new=made.kv_len.data_ptr()) == 1 and ev(keep=g + 2) == 1
    assert lib.mk_paged_prefix_attn(c.h, 0, ref, None, g, 1024, 0.1, g, 1024, None, None) == 1
    for n, cu, ln in ((3, g, g), (-1, g, g), (1, 0, g), (1, g, 0), (1, g + 2, g)):
        p = K.MkPagedPrefix(n, cu, ln)
        assert lib.mk_paged_prefix_attn(c.h, 0, ref, ctypes.byref(p), g, 1024, 0.1, g, 1024, None, None) == 1
    with pytest.raises(ValueError):
        K.PagedMass(c, torch.zeros(1, 2, 3, 4, device=DEV))
    other = Made("e4m3", 32, 2, 4, [40], 5)
    for call in (lambda: c.decode_attn_mass(0, b, torch.zeros(2, 8, 128, dtype=torch.bfloat16, device=DEV), K.PagedMass(other.c)),
                 lambda: c.evict(0, b, m, _i32([4])), lambda: c.evict(0, b, m, _i32([4, 4]), kept=_i32([1, 2])),
                 lambda: c.prefill_mass(0, two, torch.zeros(4, 8, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(3, 8, device=DEV), m),
                 lambda: K.PagedPrefix(_i32([0, 1, 2]), _i32([1]))):
        with pytest.raises(ValueError):
            call()
    # nothing to do
    none = K.PagedBatch(made.kv_len[:0], made.table[:0])
    assert lib.mk_paged_evict(c.h, 0, none.ref, g, g, 0, 0, g, 8, g, None) == 0
    assert c.poll_error() == (0, 0)


def test_two_handles_side_by_side():
    """Eviction and mass through two handles over pools of their own, on two streams at once."""
    a, b = Made("e4m3", 32, 2, 4, [20000], 5), Made("bf16", 32, 2, 4, [9000, 700], 6)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ms = []
    torch.cuda.synchronize()
    for made, s in zip((a, b), streams):
        with torch.cuda.stream(s):
            m = K.PagedMass(made.c)
            m.mass.uniform_(generator=_gen(4))
            ms.append((m, m.mass.clone(), [getattr(made.c, x + "_pool").view(torch.uint8).clone() for x in ("k", "v")],
                       None if made.kv == "bf16" else [getattr(made.c, x + "_scale").clone() for x in ("k", "v")]))
    torch.cuda.synchronize()
    res = []
    for made, s, (m, *_) in zip((a, b), streams, ms):
        res.append(made.c.evict(0, K.PagedBatch(made.kv_len, made.table), m, _i32([x // 3 for x in made.lens]), first=2, recent=9, stream=s))
    torch.cuda.synchronize()
    for made, (m, was, pools, scales), (new_len, kept) in zip((a, b), ms, res):
        assert made.c.poll_error() == (0, 0)
        before = {"k": pools[0], "v": pools[1]}
        if scales:
            before.update(ks=scales[0], vs=scales[1])
        _evict_check(made, before, was, m.mass, [x // 3 for x in made.lens], 2, 9, kept, new_len)
