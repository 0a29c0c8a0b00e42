"""The paged cache on the GPU, through the C ABI, against its 64-bit oracle.

Tolerances (fixed before the first run).  Appended codes: |code scale - y| <= half a step of e4m3 (relative 2^-4, and
scale 2^-10 among the subnormals) plus the fp32 rotation's 3 roundings, 3 * 2^-24 (|x1| + |x2|).  Attention: the
output's bf16 rounding, 2^-8 |want|; with A = sum_i w_i |v_i|, the weights' rounding before the value product, 2^-8 A
(bf16) or 2^-11 A (fp16, or bf16 in two parts); the logits' fp32 sums of 128 products, each off by at most
128 * 2^-24 * sum |q k| scale =: d, moving a normalised weight by at most 2 d; and 2^-18 A for the exponential, its
argument's rounding at |logit| <= 2^5 and the sums.  lse: d, plus 2^-18 for the sum, plus 2^-23 |lse|.
"""
import math

import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K
from compressed_kv_cache_vector_gb300.build import build
from oracle import paged_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
KV = {"bf16": K.MK_KV_BF16, "e4m3": K.MK_KV_E4M3}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(xs):
    return torch.tensor(xs, dtype=torch.int32, device=DEV)


class Made:
    """A cache with random contents: pages in scattered order, every slot that no sequence holds full of NaN."""

    def __init__(self, kv, P, n_kv, G, lens, seed, n_layers=1, layer=0, max_seqs=None, extra_cols=2, spread=0, n_pages=None):
        g = _gen(seed)
        self.kv, self.P, self.n_kv, self.G, self.lens, self.layer = kv, P, n_kv, G, lens, layer
        need = [-(-t // P) for t in lens]
        n_pages = n_pages or sum(need) + 4
        order = torch.randperm(n_pages, generator=g, device=DEV).tolist()
        cols = max(need + [1]) + extra_cols
        self.rows, at = [], 0
        for k in need:
            self.rows.append(order[at:at + k] + [-7] * (cols - k))     # never read: past the length
            at += k
        self.table = _i32(self.rows)
        cfg = K.make_paged_config(n_kv * G, n_kv, n_layers, P, n_pages, max_seqs or max(1, len(lens)), KV[kv])
        self.c = K.PagedKV(cfg, DEV)
        c = self.c
        for x in ("k", "v"):
            pool = getattr(c, x + "_pool")
            pool.view(torch.uint8).fill_(0x7f if kv == "e4m3" else 0xff)  # NaN everywhere
            if kv == "e4m3":
                getattr(c, x + "_scale").fill_(float("nan"))
            for row, t in zip(self.rows, lens):
                for j in range(-(-t // P)):
                    m = min(P, t - j * P)
                    y = torch.randn(n_kv, m, 128, generator=g, device=DEV)
                    if kv == "e4m3":
                        e = torch.randint(-spread, spread + 1, (n_kv,), generator=g, device=DEV).float() - 6
                        getattr(c, x + "_scale")[layer, row[j]] = torch.exp2(e)
                        pool[layer, row[j], :, :m] = (y * 64).to(pool.dtype)
                    else:
                        pool[layer, row[j], :, :m] = y.to(pool.dtype)
        self.kv_len = _i32(lens)

    def held(self, i, h):
        """K and V of one sequence and head as doubles [T, 128]."""
        out = []
        for x in ("k", "v"):
            pool, t = getattr(self.c, x + "_pool")[self.layer], self.lens[i]
            ids = torch.tensor(self.rows[i][: -(-t // self.P)], dtype=torch.long, device=DEV)
            if not len(ids):
                out.append(torch.zeros(0, 128, dtype=torch.float64, device=DEV))
                continue
            y = pool[:, h].view(torch.uint8 if self.kv == "e4m3" else torch.int16)[ids].view(pool.dtype).double()
            if self.kv == "e4m3":
                y = y * getattr(self.c, x + "_scale")[self.layer, ids, h].double()[:, None, None]
            out.append(y.reshape(-1, 128)[:t])
        return out


def _check_attention(made, q, out, lse, scale, news, causal, p_round, starts=None):
    G, at = made.G, 0
    for i, (t, m) in enumerate(zip(made.lens, news)):
        at = at if starts is None else starts[i]
        for h in range(made.n_kv):
            k, v = made.held(i, h)
            see = torch.arange(m, device=DEV) + t - m + 1 if causal else torch.full((m,), t, device=DEV)
            for g in range(G):
                qq = q[at:at + m, h * G + g].double()
                want, ls, A, big = O.attention(qq, k, v, scale, see)
                d = 2.0 ** -17 * big[:, None]
                tol = 2.0 ** -8 * want.abs() + (p_round + 2 * d + 2.0 ** -18) * A + 1e-30
                got = out[at:at + m, h * G + g].double()
                assert bool((got - want).abs().le(tol).all()), (i, h, g, float(((got - want).abs() / tol).max()))
                if lse is not None:
                    l2 = lse[at:at + m, h * G + g].double()
                    none = torch.isinf(ls)
                    assert torch.equal(torch.isinf(l2) & (l2 < 0), none), (i, h, g)
                    lt = d[:, 0] + 2.0 ** -18 + 2.0 ** -23 * ls.abs()
                    assert bool(((l2 - ls).abs().le(lt) | none).all()), (i, h, g)
        at += m


# ---- append ----------------------------------------------------------------------------------------------------------

def _append_oracle(state, kv, P, row, start, y):
    """Applies an append of y (double [m, heads, 128]) to {page: (codes, scale) per head} of one tensor."""
    for j in range(start // P, (start + y.shape[0] - 1) // P + 1):
        a, b = max(start, j * P), min(start + y.shape[0], (j + 1) * P)
        for h in range(y.shape[1]):
            codes, s = state.setdefault((row[j], h), (torch.zeros(P, 128, dtype=torch.float64, device=y.device), 1.0))
            part = y[a - start:b - start, h]
            if kv == "bf16":
                codes = codes.clone()
                codes[a - j * P:b - j * P] = part.to(torch.bfloat16).double()
                state[row[j], h] = (codes, 1.0)
            else:
                state[row[j], h] = O.append_page(codes, s, part, a - j * P)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("P,n_kv,steps", [(16, 2, [[1, 5, 0], [1, 1, 1], [0, 40, 15], [1, 1, 1], [33, 1, 17]]),
                                          (32, 1, [[31, 64, 1], [1, 1, 1], [1, 1, 1], [2, 31, 33]]),
                                          (64, 3, [[130, 1, 63], [1, 1, 1], [1, 0, 2], [60, 70, 1]])])
def test_append_over_several_calls_is_exact_without_rotation(kv, P, n_kv, steps):
    n, G = 3, 2
    total = [sum(s[i] for s in steps) for i in range(n)]
    made = Made(kv, P, n_kv, G, total, 5)
    c, g = made.c, _gen(77)
    before = {x: getattr(c, x + "_pool").view(torch.uint8).clone() for x in ("k", "v")}
    want = {"k": {}, "v": {}}
    have = [0] * n
    for call, news in enumerate(steps):
        rows = sum(news)
        # sizes grow and shrink from call to call, so that pages are rescaled and also keep an older, larger scale
        mag = [1.0, 30.0, 0.2, 300.0, 2.0][call % 5]
        k = (mag * torch.randn(rows, n_kv, 128, generator=g, device=DEV)).to(torch.bfloat16)
        v = (torch.randn(rows, n_kv, 128, generator=g, device=DEV) * mag / 7).to(torch.bfloat16)
        cu = [0]
        for i in range(n):
            cu.append(cu[-1] + news[i])
            have[i] += news[i]
            y = slice(cu[i], cu[i + 1])
            if news[i]:
                for x, t in (("k", k), ("v", v)):
                    _append_oracle(want[x], kv, P, made.rows[i], have[i] - news[i], t[y].double())
        b = K.PagedBatch(_i32(have), made.table, _i32(cu), max(news), rows)
        c.append(0, b, k, v)
        assert c.poll_error() == (0, 0)
        for x in ("k", "v"):
            pool = getattr(c, x + "_pool")[0]
            for (page, h), (codes, s) in want[x].items():
                i = next(i for i in range(n) if page in made.rows[i])
                held = min(P, have[i] - made.rows[i].index(page) * P)
                assert torch.equal(pool[page, h, :held].double(), codes[:held]), (call, x, page, h)
                if kv == "e4m3":
                    assert float(getattr(c, x + "_scale")[0, page, h]) == s, (call, x, page, h)
    touched = {p for p, _ in want["k"]}
    for x in ("k", "v"):                                   # pages that no sequence holds are left alone
        now = getattr(c, x + "_pool").view(torch.uint8)
        for p in range(c.cfg.n_pages):
            if p not in touched:
                assert torch.equal(now[0, p], before[x][0, p])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("rot,interleaved,given", [(128, False, False), (128, True, True), (64, False, True),
                                                   (96, True, False), (16, False, False), (48, False, True)])
def test_append_rotation(kv, rot, interleaved, given):
    P, n_kv, G, news = 32, 2, 4, [37, 1, 64]
    lens = [37 + 40, 1, 64 + 5]
    made = Made(kv, P, n_kv, G, lens, 9)
    c, g = made.c, _gen(rot)
    rows = sum(news)
    # one fused projection: q, k and v are slices of its rows
    qkv = torch.randn(rows, (G * n_kv + 2 * n_kv) * 128, generator=g, device=DEV).to(torch.bfloat16)
    q = qkv[:, : G * n_kv * 128].view(rows, G * n_kv, 128)
    k = qkv[:, G * n_kv * 128:(G + 1) * n_kv * 128].view(rows, n_kv, 128)
    v = qkv[:, (G + 1) * n_kv * 128:].view(rows, n_kv, 128)
    base = 10000.0
    table = K.rope_table(300, rot, base)
    pos = torch.cat([torch.arange(t - m, t, device=DEV) for t, m in zip(lens, news)])
    if given:
        pos = (pos * 3 + 11) % 300
    cu = [0, 37, 38, 102]
    b = K.PagedBatch(made.kv_len, made.table, _i32(cu), 64, rows)
    qo = c.append(0, b, k, v, rope=K.Rope(table, rot, interleaved, pos.int() if given else None), q=q)
    assert c.poll_error() == (0, 0)
    # the table against the definition: half a step of fp32 at 1, plus the 64-bit functions'
    ang = torch.arange(300, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    assert float((table[:, : rot // 2].cpu().double() - ang.cos()).abs().max()) < 2.0 ** -24
    size = q.double().abs().amax() * 2
    want = O.rotate(q.double(), pos, table, rot, interleaved)
    assert bool((qo.double() - want).abs().le(2.0 ** -8 * want.abs() + 3 * 2.0 ** -24 * size).all())
    assert torch.equal(qo[..., rot:], q[..., rot:])
    kk = O.rotate(k.double(), pos, table, rot, interleaved)
    top = k.double().abs().amax() * 2
    for i in range(3):
        for h in range(n_kv):
            for name, src in (("k", kk), ("v", v.double())):
                for s in range(news[i]):
                    p = lens[i] - news[i] + s
                    page = made.rows[i][p // P]
                    got = getattr(c, name + "_pool")[0, page, h, p % P].double()
                    y = src[cu[i] + s, h]
                    err = 3 * 2.0 ** -24 * top
                    if kv == "bf16":
                        tol = 2.0 ** -8 * y.abs() + err
                    else:
                        sc = float(getattr(c, name + "_scale")[0, page, h])
                        got = got * sc
                        tol = torch.maximum(2.0 ** -4 * y.abs(), torch.tensor(sc * 2.0 ** -10, device=DEV)) + err
                    assert bool((got - y).abs().le(tol).all()), (i, h, name, s)


def test_append_one_token_each_equals_a_batch_with_offsets_and_repeats_are_identical():
    for kv in ("bf16", "e4m3"):
        lens = [1, 16, 17, 100, 33]
        res = []
        for form in range(3):
            made = Made(kv, 16, 2, 2, lens, 3)
            g = _gen(4)
            k, v = (torch.randn(5, 2, 128, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
            cu = None if form == 0 else _i32([0, 1, 2, 3, 4, 5])
            b = K.PagedBatch(made.kv_len, made.table, cu, 1 if form < 2 else 4, 5)
            made.c.append(0, b, k, v, rope=K.Rope(K.rope_table(128, 128), 128))
            if form == 2:
                made.c.append(0, b, k, v, rope=K.Rope(K.rope_table(128, 128), 128))     # the same again
            assert made.c.poll_error() == (0, 0)
            res.append([made.c.k_pool.view(torch.uint8).clone(), made.c.v_pool.view(torch.uint8).clone()]
                       + ([made.c.k_scale.nan_to_num(-1.0), made.c.v_scale.nan_to_num(-1.0)] if kv == "e4m3" else []))
        for other in res[1:]:
            assert all(torch.equal(a, b) for a, b in zip(res[0], other))


def test_append_infinities_nan_zeros_and_tiny_values():
    made = Made("e4m3", 16, 1, 1, [16], 3)
    k = torch.randn(16, 1, 128, generator=_gen(1), device=DEV).clamp(-2, 2)
    k[3, 0, 5], k[3, 0, 6], k[4, 0, 7], k[0, 0, 0] = math.inf, -math.inf, math.nan, 2.0
    v = torch.zeros(16, 1, 128, device=DEV)
    b = K.PagedBatch(_i32([16]), made.table, _i32([0, 16]), 16, 16)
    made.c.append(0, b, k.to(torch.bfloat16), v.to(torch.bfloat16))
    page = made.rows[0][0]
    got = made.c.k_pool[0, page, 0].double()
    assert float(made.c.k_scale[0, page, 0]) == 2.0 ** -7             # 448 * 2^-8 = 1.75 < 2
    assert float(got[3, 5]) == 448 and float(got[3, 6]) == -448 and math.isnan(float(got[4, 7]))
    assert int(torch.isnan(got).sum()) == 1
    assert float(made.c.v_scale[0, page, 0]) == 2.0 ** -64 and not bool(made.c.v_pool[0, page, 0].float().any())
    v[:] = 1e-30
    made.c.append(0, b, k.to(torch.bfloat16), v.to(torch.bfloat16))
    assert float(made.c.v_scale[0, page, 0]) == 2.0 ** -64 and not bool(made.c.v_pool[0, page, 0].float().any())


def test_append_leaves_padding_rows_and_other_layers():
    made = Made("bf16", 16, 2, 2, [20, 9], 3, n_layers=2, layer=1)
    other = made.c.k_pool[0].view(torch.int16).clone()
    g = _gen(2)
    k, v = (torch.randn(40, 2, 128, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(40, 4, 128, generator=g, device=DEV).to(torch.bfloat16)
    qo = torch.full_like(q, 7.0)
    b = K.PagedBatch(made.kv_len, made.table, _i32([0, 20, 29]), 20, 40)
    made.c.append(1, b, k, v, q=q, q_out=qo)
    assert made.c.poll_error() == (0, 0)
    assert torch.equal(qo[:29], q[:29]) and bool((qo[29:] == 7).all())
    assert torch.equal(made.c.k_pool[0].view(torch.int16), other)
    for i, (t, r0) in enumerate(((20, 0), (9, 20))):
        for h in range(2):
            kk, vv = made.held(i, h)
            assert torch.equal(kk, k[r0:r0 + t, h].double()) and torch.equal(vv, v[r0:r0 + t, h].double())


# ---- attention -------------------------------------------------------------------------------------------------------

LENS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 130, 257, 700, 5]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("P,n_kv,G", [(16, 2, 4), (32, 1, 8), (64, 3, 1), (16, 1, 2), (64, 8, 4), (32, 2, 1)])
def test_decode_ragged(kv, P, n_kv, G):
    made = Made(kv, P, n_kv, G, LENS, 100 + P + G, n_layers=2, layer=1)
    q = (2 * torch.randn(len(LENS), n_kv * G, 128, generator=_gen(G), device=DEV)).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table)
    out, lse = made.c.decode_attn(1, b, q, lse=True)
    assert made.c.poll_error() == (0, 0)
    _check_attention(made, q, out, lse, 128 ** -0.5, [1] * len(LENS), True, 2.0 ** -11)
    assert not bool(out[0].any())
    out2, lse2 = made.c.decode_attn(1, b, q, lse=True)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16)) and torch.equal(lse, lse2)   # the same every time


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("P,n_kv,G,T", [(16, 1, 8, 20001), (32, 2, 4, 50000), (64, 8, 1, 9999)])
def test_decode_long(kv, P, n_kv, G, T):
    lens = [T, 3]
    made = Made(kv, P, n_kv, G, lens, T)
    q = torch.randn(2, n_kv * G, 128, generator=_gen(1), device=DEV).to(torch.bfloat16)
    out, lse = made.c.decode_attn(0, K.PagedBatch(made.kv_len, made.table), q, lse=True)
    assert made.c.poll_error() == (0, 0)
    _check_attention(made, q, out, lse, 128 ** -0.5, [1, 1], True, 2.0 ** -11)


@pytest.mark.parametrize("spread", [10, 30])
def test_attention_with_scales_far_apart(spread):
    """Pages whose K and V scales differ by up to 2^60: a page's weights and its values' size are independent."""
    lens = [300, 64, 17]
    made = Made("e4m3", 16, 2, 2, lens, spread, spread=spread)
    made.c.k_scale.copy_(torch.where(torch.isnan(made.c.k_scale), made.c.k_scale, torch.full_like(made.c.k_scale, 2.0 ** -6)))
    q = torch.randn(3, 4, 128, generator=_gen(1), device=DEV).to(torch.bfloat16)
    out, lse = made.c.decode_attn(0, K.PagedBatch(made.kv_len, made.table), q, lse=True)
    _check_attention(made, q, out, lse, 128 ** -0.5, [1, 1, 1], True, 2.0 ** -11)
    news = [40, 64, 3]
    q = torch.randn(107, 4, 128, generator=_gen(2), device=DEV).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table, _i32([0, 40, 104, 107]), 64, 107)
    out, lse = made.c.prefill_attn(0, b, q, lse=True)
    assert made.c.poll_error() == (0, 0)
    _check_attention(made, q, out, lse, 128 ** -0.5, news, True, 2.0 ** -11)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attention_with_one_dominant_token(kv):
    """A first token with nearly all of the weight, as attention sinks have it, and a long flat rest whose many small
    weights must not be lost; and logits of several hundred."""
    made = Made(kv, 16, 1, 4, [30000], 8)
    c, row = made.c, made.rows[0]
    u = torch.zeros(128, device=DEV)
    u[0] = 1.0
    for j, p in enumerate(row[: 30000 // 16]):
        if kv == "e4m3":
            c.k_scale[0, p] = 0.125
        c.k_pool[0, p, 0] = 0
    c.k_pool[0, row[0], 0, 0] = (u * (8 / 0.125 if kv == "e4m3" else 8)).to(c.k_pool.dtype)
    for size in (8.0, 16.0, 600.0):
        q = torch.zeros(1, 4, 128, device=DEV)
        q[:, :, 0] = size
        q = q.to(torch.bfloat16)
        out, lse = c.decode_attn(0, K.PagedBatch(made.kv_len, made.table), q, lse=True)
        _check_attention(made, q, out, lse, 128 ** -0.5, [1], True, 2.0 ** -11)
        qq = q.expand(5, 4, 128).contiguous()
        b = K.PagedBatch(made.kv_len, made.table, _i32([0, 5]), 5, 5)
        out, lse = c.prefill_attn(0, b, qq, lse=True)
        _check_attention(made, qq, out, lse, 128 ** -0.5, [5], True, 2.0 ** -8 if kv == "bf16" else 2.0 ** -11)
    assert c.poll_error() == (0, 0)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("P,n_kv,G", [(16, 2, 4), (32, 1, 8), (64, 3, 1), (16, 2, 2)])
def test_prefill_ragged(kv, causal, P, n_kv, G):
    """Queries before and past tile borders, contexts of every residue, no new tokens, an empty context, and (causal)
    more queries than keys: their first rows see nothing."""
    lens = [0, 1, 40, 129, 200, 64, 333, 12, 5, 700]
    news = [3, 1, 0, 129, 7, 64, 130, 33, 2, 257]
    made = Made(kv, P, n_kv, G, lens, 50 + P + G)
    rows = sum(news)
    cu = [0]
    for m in news:
        cu.append(cu[-1] + m)
    q = (1.5 * torch.randn(rows, n_kv * G, 128, generator=_gen(G), device=DEV)).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table, _i32(cu), max(news), rows)
    out, lse = made.c.prefill_attn(0, b, q, causal=causal, scale=0.11, lse=True)
    assert made.c.poll_error() == (0, 0)
    _check_attention(made, q, out, lse, 0.11, news, causal, 2.0 ** -8 if kv == "bf16" else 2.0 ** -11)
    assert not bool(out[:3].any())
    out2, lse2 = made.c.prefill_attn(0, b, q, causal=causal, scale=0.11, lse=True)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("news,lens,G", [([600], [600], 4), ([513], [4100], 4), ([2, 4], [6000, 3333], 4), ([300], [1500], 1),
                                         ([9], [20000], 8), ([40, 900, 33, 500, 3, 1200], [3000, 2500, 4000, 700, 2600, 1200], 4)])
def test_prefill_longer(kv, news, lens, G):
    made = Made(kv, 32, 2, G, lens, 7)
    rows = sum(news)
    cu = [0]
    for m in news:
        cu.append(cu[-1] + m)
    q = torch.randn(rows, 2 * G, 128, generator=_gen(3), device=DEV).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table, _i32(cu), max(news), rows)
    out, lse = made.c.prefill_attn(0, b, q, lse=True)
    assert made.c.poll_error() == (0, 0)
    _check_attention(made, q, out, lse, 128 ** -0.5, news, True, 2.0 ** -8 if kv == "bf16" else 2.0 ** -11)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_strided_rows_padding_and_streams(kv):
    lens, news = [50, 90, 33], [4, 20, 1]
    made = Made(kv, 16, 2, 2, lens, 6)
    wide = torch.randn(40, 10 * 128, generator=_gen(5), device=DEV).to(torch.bfloat16)
    q = wide[:, 128:128 * 5].view(40, 4, 128)
    res = torch.full((40, 6, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((40, 4), 5.0, device=DEV)
    b = K.PagedBatch(made.kv_len, made.table, _i32([0, 4, 24, 25]), 20, 40)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    made.c.prefill_attn(0, b, q, out=res[:, 1:5], lse=lse, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    _check_attention(made, q, res[:, 1:5], lse, 128 ** -0.5, news, True, 2.0 ** -8 if kv == "bf16" else 2.0 ** -11)
    assert bool((res[25:] == 3).all()) and bool((res[:, 0] == 3).all()) and bool((res[:, 5] == 3).all())
    assert bool((lse[25:] == 5).all())
    res.fill_(3.0)
    lse.fill_(5.0)
    b = K.PagedBatch(made.kv_len, made.table, n_tokens=40)          # padded rows behind the three sequences
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        made.c.decode_attn(0, b, q, out=res[:, 1:5], lse=lse)
    torch.cuda.current_stream().wait_stream(s)
    _check_attention(made, q, res[:, 1:5], lse, 128 ** -0.5, [1, 1, 1], True, 2.0 ** -11)
    assert bool((res[3:] == 3).all()) and bool((res[:, 0] == 3).all()) and bool((lse[3:] == 5).all())
    b = K.PagedBatch(made.kv_len, made.table, _i32([2, 3, 3, 4]), 1, 40)   # the second sequence has no token
    res.fill_(3.0)
    made.c.decode_attn(0, b, q, out=res[:, 1:5], lse=lse)
    assert made.c.poll_error() == (0, 0)
    _check_attention(made, q, res[:, 1:5], None, 128 ** -0.5, [1, 0, 1], True, 2.0 ** -11, starts=[2, 3, 3])
    assert bool((res[:2] == 3).all()) and bool((res[4:] == 3).all())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_run_of_the_operators_eager_and_captured(kv):
    """A prompt, then decode steps: append with rotation and attention, as a serving loop runs them; the same steps as
    a captured graph replayed with the lengths advanced on the device, and a second graph of the same handle."""
    P, n_kv, G, first, steps = 16, 2, 4, [70, 33], 20
    lens = [f + steps for f in first]
    table_rope = K.rope_table(256, 128)
    g = _gen(21)
    toks = {x: torch.randn(2, 120, h, 128, generator=g, device=DEV).to(torch.bfloat16)
            for x, h in (("q", n_kv * G), ("k", n_kv), ("v", n_kv))}

    def start():
        made = Made(kv, P, n_kv, G, lens, 4)
        rope = K.Rope(table_rope, 128)
        kv_len = _i32(first)
        rows = sum(first)
        pick = lambda x: torch.cat([toks[x][0, :first[0]], toks[x][1, :first[1]]])  # noqa: E731
        b = K.PagedBatch(kv_len, made.table, _i32([0, first[0], rows]), max(first), rows)
        q = made.c.append(0, b, pick("k"), pick("v"), rope=rope, q=pick("q"))
        o = made.c.prefill_attn(0, b, q)
        return made, rope, kv_len, q, o

    made, rope, kv_len, q, o = start()
    made.lens = list(first)
    _check_attention(made, q, o, None, 128 ** -0.5, first, True, 2.0 ** -8 if kv == "bf16" else 2.0 ** -11)
    want = []
    b = K.PagedBatch(kv_len, made.table)
    for t in range(steps):
        x = {n: torch.stack([toks[n][i, first[i] + t] for i in range(2)]) for n in toks}
        kv_len.add_(1)
        q = made.c.append(0, b, x["k"], x["v"], rope=rope, q=x["q"])
        o = made.c.decode_attn(0, b, q)
        want.append(o.clone())
        if t in (0, 7, steps - 1):
            made.lens = [f + t + 1 for f in first]
            _check_attention(made, q, o, None, 128 ** -0.5, [1, 1], True, 2.0 ** -11)
    assert made.c.poll_error() == (0, 0)

    made, rope, kv_len, _, _ = start()
    b = K.PagedBatch(kv_len, made.table)
    x = {n: torch.zeros(2, h, 128, dtype=torch.bfloat16, device=DEV) for n, h in (("q", n_kv * G), ("k", n_kv), ("v", n_kv))}
    out = torch.zeros(2, n_kv * G, 128, dtype=torch.bfloat16, device=DEV)
    qo = torch.zeros_like(out)
    graphs = []
    torch.cuda.synchronize()
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            kv_len.add_(1)
            made.c.append(0, b, x["k"], x["v"], rope=rope, q=x["q"], q_out=qo)
            made.c.decode_attn(0, b, qo, out=out)
        graphs.append(gr)
    for t in range(steps):
        for n in toks:
            x[n].copy_(torch.stack([toks[n][i, first[i] + t] for i in range(2)]))
        graphs[t % 2].replay()
        assert torch.equal(out.view(torch.int16), want[t].view(torch.int16)), t
    assert made.c.poll_error() == (0, 0)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_offsets_past_32_bits(kv):
    """A pool of more than 2^32 bytes (and, in bf16, page offsets past 2^31 elements), used at its end."""
    P, n_kv, G = 64, 8, 2
    n_pages = (1 << 32) // (n_kv * P * 128 * (1 if kv == "e4m3" else 2)) + 70
    made = Made(kv, P, n_kv, G, [130, 70], 2, n_pages=n_pages)
    c = made.c
    # the same contents moved to the last pages of the pool
    last = list(range(n_pages - 5, n_pages))
    old = made.rows[0][:3] + made.rows[1][:2]
    for x in ("k", "v"):
        pool = getattr(c, x + "_pool").view(torch.uint8)
        keep = [pool[0, p].clone() for p in old]
        sc = [getattr(c, x + "_scale")[0, p].clone() for p in old] if kv == "e4m3" else None
        for n, p in enumerate(last):
            pool[0, p] = keep[n]
            if sc:
                getattr(c, x + "_scale")[0, p] = sc[n]
    made.rows = [last[:3], last[3:] + [-7]]
    made.table = _i32(made.rows)
    q = torch.randn(2, n_kv * G, 128, generator=_gen(3), device=DEV).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table)
    out, lse = c.decode_attn(0, b, q, lse=True)
    _check_attention(made, q, out, lse, 128 ** -0.5, [1, 1], True, 2.0 ** -11)
    k, v = (torch.randn(100, n_kv, 128, generator=_gen(9), device=DEV).to(torch.bfloat16) for _ in range(2))
    b = K.PagedBatch(made.kv_len, made.table, _i32([0, 60, 100]), 60, 100)
    q = torch.randn(100, n_kv * G, 128, generator=_gen(3), device=DEV).to(torch.bfloat16)
    c.append(0, b, k, v)
    out, lse = c.prefill_attn(0, b, q, lse=True)
    assert c.poll_error() == (0, 0)
    _check_attention(made, q, out, lse, 128 ** -0.5, [60, 40], True, 2.0 ** -8 if kv == "bf16" else 2.0 ** -11)


# ---- refusals and device errors --------------------------------------------------------------------------------------

def test_refusals_before_any_launch():
    made = Made("e4m3", 16, 2, 2, [20, 9], 3)
    c = made.c
    k = torch.randn(3, 2, 128, device=DEV).to(torch.bfloat16)
    q = torch.randn(3, 4, 128, device=DEV).to(torch.bfloat16)
    one = K.PagedBatch(made.kv_len, made.table)
    many = K.PagedBatch(made.kv_len, made.table, _i32([0, 1, 3]), 2, 3)
    before = c.k_pool.view(torch.uint8).clone()
    for call in (lambda: c.decode_attn(0, many, q),                               # more than one token per sequence
                 lambda: c.decode_attn(1, one, q), lambda: c.decode_attn(-1, one, q),   # no such layer
                 lambda: c.decode_attn(0, one, q, scale=float("nan")), lambda: c.decode_attn(0, one, q, scale=float("inf")),
                 lambda: c.prefill_attn(0, K.PagedBatch(made.kv_len, made.table, None, 2), q),   # offsets are missing
                 lambda: c.append(0, one, k.view(-1)[4:516].view(2, 2, 128), k),    # 8-byte aligned
                 lambda: c.append(0, one, k, k, rope=K.Rope(torch.zeros(4, 24, device=DEV), 24))):
        with pytest.raises(K.MosaicKVError) as e:
            call()
        assert e.value.status == 1
    short = K.Rope(K.rope_table(64, 128), 128, positions=_i32([0]))
    for call in (lambda: c.append(0, one, k, k, rope=short), lambda: c.decode_attn(0, one, q.float()), lambda: c.decode_attn(0, one, q[:1]),
                 lambda: c.decode_attn(0, one, q[:, :3]), lambda: c.append(0, one, k, k, q_out=q),
                 lambda: c.append(0, one, k.transpose(1, 2), k), lambda: c.decode_attn(0, one, q.cpu()),
                 lambda: c.prefill_attn(0, many, q, lse=torch.zeros(2, 4, device=DEV)),
                 lambda: K.PagedBatch(made.kv_len.long(), made.table),
                 lambda: K.PagedBatch(made.kv_len, made.table, _i32([0, 1]), 1, 1)):
        with pytest.raises(ValueError):
            call()
    assert torch.equal(c.k_pool.view(torch.uint8), before)
    empty = K.PagedBatch(_i32([]), torch.zeros(0, 3, dtype=torch.int32, device=DEV))
    assert c.decode_attn(0, empty, q[:0]).shape == (0, 4, 128)
    assert c.poll_error() == (0, 0)


@pytest.mark.parametrize("what", ["page", "negative page", "length", "negative length", "offsets", "position"])
def test_device_errors_are_recorded_and_sticky(what):
    """Values that only the device sees: the error word is set, later calls leave their output, clearing mends it."""
    made = Made("e4m3", 16, 1, 2, [40, 20], 3)
    c = made.c
    k = torch.randn(4, 1, 128, device=DEV).to(torch.bfloat16)
    q = torch.randn(4, 2, 128, device=DEV).to(torch.bfloat16)
    table, kv_len, cu, rope, detail = made.table.clone(), made.kv_len.clone(), _i32([0, 2, 4]), None, 16
    if what == "page":
        table[0, 2], detail = c.cfg.n_pages, 17
    elif what == "negative page":
        table[0, 2], detail = -1, 17
    elif what == "length":
        kv_len[0] = 16 * table.shape[1] + 1
    elif what == "negative length":
        kv_len[1] = -3
    elif what == "offsets":
        cu = _i32([0, 2, 9])
    else:
        rope, detail = K.Rope(K.rope_table(30, 128), 128), 18
    b = K.PagedBatch(kv_len, table, cu, 2, 4)
    calls = [lambda: c.append(0, b, k, k, rope=rope)]
    if what != "position":
        calls.append(lambda: c.prefill_attn(0, b, q))
        if what != "offsets":
            calls.append(lambda: c.decode_attn(0, K.PagedBatch(kv_len, table), q))
    good = K.PagedBatch(made.kv_len, made.table)
    out = torch.zeros_like(q)
    for call in calls:
        call()
        assert c.poll_error() == (5, detail)
        out.fill_(9.0)
        c.decode_attn(0, good, q, out=out)
        assert bool((out == 9).all())
        c.clear_error()
        assert c.poll_error() == (0, 0)
        c.decode_attn(0, good, q, out=out)
        assert not bool((out[:2] == 9).any()) and c.poll_error() == (0, 0)


def test_the_handle_keeps_its_device_and_two_handles_run_side_by_side():
    a, b = Made("e4m3", 16, 2, 4, [3000, 700], 1), Made("bf16", 32, 2, 4, [1500, 2200], 2)
    q = torch.randn(2, 8, 128, generator=_gen(2), device=DEV).to(torch.bfloat16)
    ba, bb = K.PagedBatch(a.kv_len, a.table), K.PagedBatch(b.kv_len, b.table)
    wa, wb = a.c.decode_attn(0, ba, q).clone(), b.c.decode_attn(0, bb, q).clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(20):
        outs.append((a.c.decode_attn(0, ba, q, stream=s1), b.c.decode_attn(0, bb, q, stream=s2)))
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(x.view(torch.int16), wa.view(torch.int16)) and torch.equal(y.view(torch.int16), wb.view(torch.int16))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attention_of_zero_rows_zero_pages_and_zero_or_negative_scale(kv):
    made = Made(kv, 16, 2, 2, [150, 33], 11)
    c, rows = made.c, made.rows
    for p in rows[0][:4]:
        c.k_pool[0, p].view(torch.uint8).zero_()
        if kv == "e4m3":
            c.k_scale[0, p] = 2.0 ** -64
    for p in rows[0][2:7]:
        c.v_pool[0, p].view(torch.uint8).zero_()
        if kv == "e4m3":
            c.v_scale[0, p] = 2.0 ** -64
    q = torch.randn(60, 4, 128, generator=_gen(8), device=DEV).to(torch.bfloat16)
    q[3:7] = 0
    q[50:52, 1] = 0
    b = K.PagedBatch(made.kv_len, made.table, _i32([0, 40, 60]), 40, 60)
    one = K.PagedBatch(made.kv_len, made.table)
    for scale in (0.0, -0.1, 128 ** -0.5):
        for causal in (True, False):
            out, lse = c.prefill_attn(0, b, q, causal=causal, scale=scale, lse=True)
            _check_attention(made, q, out, lse, scale, [40, 20], causal, 2.0 ** -8 if kv == "bf16" else 2.0 ** -11)
        qq = q[2:4].contiguous()
        out, lse = c.decode_attn(0, one, qq, scale=scale, lse=True)
        _check_attention(made, qq, out, lse, scale, [1, 1], True, 2.0 ** -11)
    assert c.poll_error() == (0, 0)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_nan_key_reaches_only_the_queries_that_see_it(kv):
    lens, at = [600], 300
    made = Made(kv, 16, 2, 4, lens, 12)
    c = made.c
    q = torch.randn(600, 8, 128, generator=_gen(4), device=DEV).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table, _i32([0, 600]), 600, 600)
    want, wl = c.prefill_attn(0, b, q, lse=True)
    nan = 0x7f if kv == "e4m3" else 0xff
    c.k_pool[0, made.rows[0][at // 16], 1, at % 16].view(torch.uint8).fill_(nan)        # head 1, token 300
    out, lse = c.prefill_attn(0, b, q, lse=True)
    assert torch.equal(out[:at], want[:at]) and torch.equal(lse[:at], wl[:at])
    assert torch.equal(out[:, :4], want[:, :4]) and torch.equal(lse[:, :4], wl[:, :4])
    assert bool(torch.isnan(out[at:, 4:]).all()) and bool(torch.isnan(lse[at:, 4:]).all())
    one = K.PagedBatch(_i32([at]), made.table)
    assert not bool(torch.isnan(c.decode_attn(0, one, q[:1])).any())
    one = K.PagedBatch(_i32([at + 1]), made.table)
    assert bool(torch.isnan(c.decode_attn(0, one, q[:1])[:, 4:]).all())
    assert c.poll_error() == (0, 0)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("P,n_kv,G", [(16, 2, 4), (32, 1, 8), (64, 3, 1), (16, 2, 2)])
def test_prefill_of_few_tokens(kv, causal, P, n_kv, G):
    """Up to 16 rows a kv head, partly filled, empty contexts, no tokens, more tokens than keys, contexts that end at
    and around the borders of pages and chunks, and a long one split over CTAs."""
    top = 16 // G
    lens = [0, 1, 2, 15, 16, 17, 31, 33, 64, 130, 700, 5000, 40, top - 1]
    news = [min(m, top) for m in (1, top, 1, 2, top, 3, 1, top - 1, top, 2, top // 2, top, 0, top)]
    made = Made(kv, P, n_kv, G, lens, 70 + P + G)
    rows = sum(news)
    cu = [0]
    for m in news:
        cu.append(cu[-1] + m)
    q = (1.5 * torch.randn(rows + 3, n_kv * G, 128, generator=_gen(G), device=DEV)).to(torch.bfloat16)
    out = torch.full_like(q, 4.0)
    lse = torch.full((rows + 3, n_kv * G), 4.0, device=DEV)
    b = K.PagedBatch(made.kv_len, made.table, _i32(cu), top, rows + 3)
    made.c.prefill_attn(0, b, q, causal=causal, out=out, lse=lse)
    assert made.c.poll_error() == (0, 0)
    _check_attention(made, q, out, lse, 128 ** -0.5, news, causal, 2.0 ** -11)
    assert bool((out[rows:] == 4).all()) and bool((lse[rows:] == 4).all())
    again = made.c.prefill_attn(0, b, q, causal=causal, out=torch.full_like(q, 4.0))
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


def test_prefill_of_few_and_of_many_tokens_agree():
    """The two kernels behind prefill_attn on the same tokens: 4 a sequence as a batch of at most 4, and of at most 5."""
    for kv in ("bf16", "e4m3"):
        made = Made(kv, 32, 2, 4, [900, 4, 333], 17)
        q = torch.randn(12, 8, 128, generator=_gen(2), device=DEV).to(torch.bfloat16)
        cu = _i32([0, 4, 8, 12])
        few, fl = made.c.prefill_attn(0, K.PagedBatch(made.kv_len, made.table, cu, 4, 12), q, lse=True)
        many, ml = made.c.prefill_attn(0, K.PagedBatch(made.kv_len, made.table, cu, 5, 12), q, lse=True)
        assert made.c.poll_error() == (0, 0)
        for out, lse in ((few, fl), (many, ml)):
            _check_attention(made, q, out, lse, 128 ** -0.5, [4, 4, 4], True, 2.0 ** -8 if kv == "bf16" else 2.0 ** -11)
