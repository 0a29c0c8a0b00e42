"""The paged cache where a call meets a limit of its kernels: contexts so long that waits inside a kernel last, numbers
that are not finite, scales far apart, errors of one sequence beside good ones, lengths that go back.

The bounds are those of test_gpu_paged.py; a test that needs another one derives it beside its inputs.
"""
import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K
from compressed_kv_cache_vector_gb300.build import build
from oracle import paged_oracle as O
from tests.test_gpu_paged import DEV, KV, Made, _append_oracle, _check_attention, _gen, _i32

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


# ---- errors of one sequence beside good ones -------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("what", ["page", "length"])
def test_a_bad_sequence_leaves_the_others_of_its_call_complete(kv, what):
    """An append of many waves of CTAs, whose first ones meet the error, and attention of both kinds behind it."""
    P, n_kv, G, n, m = 16, 4, 2, 40, 512
    cfg = K.make_paged_config(n_kv * G, n_kv, 1, P, n * m // P + 2, n, KV[kv])
    g = _gen(3)
    table = torch.randperm(n * m // P, generator=g, device=DEV).int().view(n, m // P).contiguous()
    k, v = (torch.randn(n * m, n_kv, 128, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(n * m, n_kv * G, 128, generator=g, device=DEV).to(torch.bfloat16)
    lens, cu = [m] * n, [m * i for i in range(n + 1)]
    rope = K.Rope(K.rope_table(m, 128), 128)
    good = torch.tensor([i for i in range(n) if i != 1], device=DEV)
    pages, rows = table[good].flatten().long(), (good[:, None] * m + torch.arange(m, device=DEV)).flatten()

    def run(kv_len, tab):
        offsets = _i32(cu)
        c = K.PagedKV(cfg, DEV)
        b, res, states = K.PagedBatch(kv_len, tab, offsets, m, n * m), [], []

        def done(*outs):
            states.append(c.poll_error())
            if states[-1][0]:
                c.clear_error()
            res.extend(outs)

        qo = c.append(0, b, k, v, rope=rope, q=q, q_out=torch.zeros_like(q))
        done(qo[rows], *(getattr(c, x + "_pool")[0].view(torch.uint8)[pages].clone() for x in ("k", "v")),
             *([c.k_scale[0, pages], c.v_scale[0, pages]] if kv == "e4m3" else []))
        # The split over CTAs depends on the lengths of all sequences: attention is compared with the oracle.
        for per, call in ((m, c.prefill_attn), (1, c.decode_attn), (2, c.prefill_attn)):
            b = K.PagedBatch(kv_len, tab, offsets if per == m else _i32([per * i for i in range(n + 1)]), per, per * n)
            o, lse = torch.full_like(q[: per * n], float("nan")), torch.full((per * n, n_kv * G), float("nan"), device=DEV)
            call(0, b, qo[: per * n], out=o, lse=lse)
            done()
            fine = torch.isfinite(o.float()).all(dim=2) & torch.isfinite(lse)
            assert bool(fine.view(n, -1)[good].all())
            for i in (0, 2, 17, n - 1):
                for h in range(n_kv):
                    kk, vv = (p[0, :, h].view(torch.uint8 if kv == "e4m3" else torch.int16)[table[i].long()].view(p.dtype)
                              .double() for p in (c.k_pool, c.v_pool))
                    if kv == "e4m3":
                        kk, vv = (y * s[0, table[i].long(), h].double()[:, None, None]
                                  for y, s in ((kk, c.k_scale), (vv, c.v_scale)))
                    see = torch.arange(per, device=DEV) + m - per + 1
                    for x in range(h * G, (h + 1) * G):
                        at = slice(i * per, (i + 1) * per)
                        w, ls, A, big = O.attention(qo[at, x].double(), kk.reshape(-1, 128), vv.reshape(-1, 128), 128 ** -0.5, see)
                        d = 2.0 ** -17 * big[:, None]
                        p_round = 2.0 ** -8 if kv == "bf16" and per == m else 2.0 ** -11
                        tol = 2.0 ** -8 * w.abs() + (p_round + 2 * d + 2.0 ** -18) * A + 1e-30
                        assert bool((o[at, x].double() - w).abs().le(tol).all()), (per, i, x)
                        assert bool((lse[at, x].double() - ls).abs().le(d[:, 0] + 2.0 ** -18 + 2.0 ** -23 * ls.abs()).all())
        return res, states

    want, states = run(_i32(lens), table)
    assert states == [(0, 0)] * 4
    if what == "page":
        table[1, 0] = 10 ** 6
    else:
        lens[1] = 16 * table.shape[1] + 1
    got, states = run(_i32(lens), table)
    assert states == [(5, 17 if what == "page" else 16)] * 4
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_an_error_keeps_later_calls_and_replays_from_working():
    P, n_kv, G = 16, 2, 2
    cfg = K.make_paged_config(n_kv * G, n_kv, 1, P, 8, 2)
    table, kv_len = _i32([[0, 1], [10 ** 6, 3]]), _i32([5, 5])
    k = torch.randn(2, n_kv, 128, device=DEV).to(torch.bfloat16)
    q = torch.randn(2, n_kv * G, 128, device=DEV).to(torch.bfloat16)
    out = torch.zeros_like(q)
    for between in ("attention", "poll"):
        c = K.PagedKV(cfg, DEV)
        table[1, 0], b = 10 ** 6, K.PagedBatch(kv_len, table)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.append(0, b, k, k)
            if between == "attention":
                c.decode_attn(0, b, q, out=out)
        out.fill_(9.0)
        gr.replay()
        torch.cuda.synchronize()
        assert bool(c.k_pool[0, 0, :, 4].float().any())               # the good sequence's token is stored
        assert bool((out == 9).all())                                 # the call behind it does nothing
        if between == "poll":
            assert c.poll_error() == (5, 17)
        table[1, 0] = 2
        c.k_pool.view(torch.uint8).zero_()
        gr.replay()
        assert not bool(c.k_pool.float().any()) and c.poll_error() == (5, 17)
        c.clear_error()
        gr.replay()
        assert bool(c.k_pool[0, 0, :, 4].float().any()) and bool(c.k_pool[0, 2, :, 4].float().any())
        assert c.poll_error() == (0, 0)


# ---- numbers that are not finite, and scales far apart ---------------------------------------------------------------

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n_nan", [0, 600, 20000, 50000])
def test_nan_logits_give_nan_however_the_tokens_are_split(kv, n_nan):
    """NaN in a query row, or in the keys of one head from the first on, which fill the chunks of whole warps and whole
    CTAs: out and lse are NaN in exactly the rows that see one, in every form of the attention."""
    lens, n_kv, G = [700, 50000], 2, 2
    made = Made(kv, 16, n_kv, G, lens, 12)
    c = made.c
    for p in made.rows[1][: n_nan // 16]:
        c.k_pool[0, p, 1].view(torch.uint8).fill_(0x7f if kv == "e4m3" else 0xff)
    for form, news in (("decode", [1, 1]), ("few", [3, 8]), ("wide", [150, 40])):
        rows = sum(news)
        q = torch.randn(rows, n_kv * G, 128, generator=_gen(4), device=DEV).to(torch.bfloat16)
        q[0, 0], q[rows - 1, 3, 77] = float("nan"), float("nan")
        want = torch.zeros(rows, n_kv * G, dtype=torch.bool, device=DEV)
        want[0, 0] = want[rows - 1, 3] = True
        want[news[0]:, 2:] |= n_nan > 0
        b = K.PagedBatch(made.kv_len, made.table, _i32([0, news[0], rows]), max(news), rows)
        for causal in (True, False):
            out, lse = c.decode_attn(0, b, q, lse=True) if form == "decode" else c.prefill_attn(0, b, q, causal, lse=True)
            assert c.poll_error() == (0, 0)
            assert torch.equal(torch.isnan(lse), want), (form, causal)
            assert torch.equal(torch.isnan(out), want[..., None].expand_as(out)), (form, causal)
            assert bool(torch.isfinite(lse[~want]).all())


@pytest.mark.parametrize("low,high", [(-64, 16), (40, 120)])
@pytest.mark.parametrize("order", ["alternating", "low first", "high first"])
def test_v_scales_at_the_limit_of_their_distance(low, high, order):
    """V scales 2^80 apart in pages next to each other, and in halves of the context, so that warps and CTAs differ.

    The bounds of test_gpu_paged.py hold for weights in fp16's normal range.  Below it a weight (times its page's V
    scale b, and 2^10 or more relative to the row's largest such product M) is off by half of fp16's smallest step,
    2^-25, so by at most 2^-35 M: with scales this far apart that is all that some tokens have.  Each multiplies its
    code, so 2^-35 max_i (p_i b_i) sum_i |code_i| comes on top, p_i the normalised weights: what is left in a channel
    where the tokens of the large scale happen to hold zeros."""
    lens, n_kv, G = [3000, 40], 2, 2
    made = Made("e4m3", 16, n_kv, G, lens, 5)
    for i, row in enumerate(made.rows):
        n = -(-lens[i] // 16)
        for j, p in enumerate(row[:n]):
            up = {"alternating": j % 2, "low first": j >= n // 2, "high first": j < n // 2}[order]
            made.c.v_scale[0, p] = 2.0 ** (high if up else low)
            m = min(16, lens[i] - 16 * j)
            made.c.v_pool[0, p, :, :m] = torch.randn(n_kv, m, 128, generator=_gen(p), device=DEV).to(made.c.v_pool.dtype)
    for form, news in (("decode", [1, 1]), ("few", [3, 8]), ("wide", [150, 40])):
        rows = sum(news)
        q = (2 * torch.randn(rows, n_kv * G, 128, generator=_gen(4), device=DEV)).to(torch.bfloat16)
        b = K.PagedBatch(made.kv_len, made.table, _i32([0, news[0], rows]), max(news), rows)
        out, lse = made.c.decode_attn(0, b, q, lse=True) if form == "decode" else made.c.prefill_attn(0, b, q, lse=True)
        assert made.c.poll_error() == (0, 0)
        for i, (t, m, r0) in enumerate(zip(lens, news, (0, news[0]))):
            see = torch.arange(m, device=DEV) + t - m + 1
            pages = torch.tensor(made.rows[i][: -(-t // 16)], device=DEV)
            for x in range(n_kv * G):
                k, v = made.held(i, x // G)
                qq, got, ls = q[r0:r0 + m, x].double(), out[r0:r0 + m, x].double(), lse[r0:r0 + m, x].double()
                want, wl, A, big = O.attention(qq, k, v, 128 ** -0.5, see)
                d = 2.0 ** -17 * big[:, None]
                b_tok = made.c.v_scale[0, pages, x // G].double().repeat_interleave(16)[:t]
                hid = torch.arange(t, device=DEV)[None, :] >= see[:, None]
                p = torch.exp(qq @ k.T * 128 ** -0.5 - wl[:, None]).masked_fill(hid, 0)
                codes = (~hid).double() @ (v / b_tok[:, None]).abs()
                tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * d + 2.0 ** -18) * A
                tol += 2.0 ** -35 * (p * b_tok).amax(dim=1, keepdim=True) * codes
                assert bool((got - want).abs().le(tol).all()), (form, i, x, float(((got - want).abs() / tol).max()))
                assert bool((ls - wl).abs().le(d[:, 0] + 2.0 ** -18 + 2.0 ** -23 * wl.abs()).all()), (form, i, x)


# ---- other streams ---------------------------------------------------------------------------------------------------

def test_memory_that_a_queued_call_reads_is_not_handed_out_again():
    """Batch and rotation dropped while the call that reads them waits behind another kernel of its stream."""
    made = Made("bf16", 16, 2, 2, [50, 90, 33], 6)
    k, v = (torch.randn(3, 2, 128, generator=_gen(i), device=DEV).to(torch.bfloat16) for i in (1, 2))
    q = torch.randn(3, 4, 128, generator=_gen(3), device=DEV).to(torch.bfloat16)
    table = K.rope_table(100, 128)
    qo = torch.empty_like(q)
    want = made.c.append(0, K.PagedBatch(made.kv_len, made.table), k, v, rope=K.Rope(table, 128), q=q)
    o = made.c.decode_attn(0, K.PagedBatch(made.kv_len, made.table), want)
    out = torch.zeros_like(o)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    made.c.k_pool[0, made.rows[0][3], :, 1] = 0            # the first sequence's token is stored anew
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    parts = [made.kv_len.clone(), made.table.clone(), table.clone(), _i32([49, 89, 32])]
    torch.cuda.current_stream().synchronize()
    spec = [(x.shape, x.dtype, x.data_ptr()) for x in parts]
    b = K.PagedBatch(parts[0], parts[1])
    made.c.append(0, b, k, v, rope=K.Rope(parts[2], 128, positions=parts[3]), q=q, q_out=qo, stream=s)
    made.c.decode_attn(0, b, qo, out=out, stream=s)
    queued = not s.query()
    del parts, b
    new = [torch.zeros(shape, dtype=dtype, device=DEV) for shape, dtype, _ in spec]      # what comes next on this stream
    assert queued and not {x.data_ptr() for x in new} & {p for _, _, p in spec}
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(qo, want) and torch.equal(out, o) and made.c.poll_error() == (0, 0)


def test_new_outputs_for_another_stream_do_not_reuse_what_this_one_still_reads():
    made = Made("bf16", 16, 2, 2, [50, 90, 33], 6)
    q = torch.randn(3, 4, 128, generator=_gen(3), device=DEV).to(torch.bfloat16)
    b = K.PagedBatch(made.kv_len, made.table)
    want = made.c.decode_attn(0, b, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    old = torch.full_like(q, 3.0)
    torch.cuda._sleep(100_000_000)
    copy = old.clone()                                     # queued behind the sleep, and then the block is free
    del old
    out, lse = made.c.decode_attn(0, b, q, lse=True, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    torch.cuda.current_stream().wait_stream(s)
    assert bool((copy == 3.0).all()) and made.c.poll_error() == (0, 0)


# ---- refusals --------------------------------------------------------------------------------------------------------

def test_word_arrays_off_their_alignment_are_refused_before_any_launch():
    made = Made("e4m3", 16, 2, 2, [50, 33], 6)
    c, lib = made.c, K.load()
    q = torch.randn(2, 4, 128, generator=_gen(3), device=DEV).to(torch.bfloat16)
    out, cu, lse = torch.full_like(q, 5.0), _i32([0, 1, 2]), torch.full((2, 4), 5.0, device=DEV)
    table = K.rope_table(64, 128)
    pos = _i32([1, 2])
    before = [c.k_pool.view(torch.uint8).clone(), c.k_scale.nan_to_num(-1.0)]

    def batch(*off):
        return K.MkPagedBatch(2, 2, 1, made.table.shape[1], cu.data_ptr() + off[0], made.kv_len.data_ptr() + off[1],
                              made.table.data_ptr() + off[2])

    def append(b, at=0):
        r = K.MkRope(table.data_ptr(), 64, 128, 0, pos.data_ptr() + at)
        return lib.mk_paged_append(c.h, 0, ref(b), ref(r), p, 512, p, 512, None, 0, None, 0, st)

    def decode(b, at=0):
        return lib.mk_paged_decode_attn(c.h, 0, ref(b), p, 512, 0.1, out.data_ptr(), 512, lse.data_ptr() + at, st)

    def prefill(b, at=0):
        return lib.mk_paged_prefill_attn(c.h, 0, ref(b), 1, p, 512, 0.1, out.data_ptr(), 512, lse.data_ptr() + at, st)

    ref, p, st = K.ctypes.byref, q.data_ptr(), K._raw_stream(c.device.index)
    for call in (append, decode, prefill):
        for by in (1, 2, 3):
            for i in range(3):
                assert call(batch(*(by if j == i else 0 for j in range(3)))) == 1
            assert call(batch(0, 0, 0), by) == 1               # positions, or lse
    assert c.poll_error() == (0, 0)
    assert torch.equal(c.k_pool.view(torch.uint8), before[0]) and torch.equal(c.k_scale.nan_to_num(-1.0), before[1])
    assert bool((out == 5).all()) and bool((lse == 5).all())
    assert [call(batch(0, 0, 0)) for call in (append, decode, prefill)] == [0, 0, 0] and c.poll_error() == (0, 0)


# ---- lengths that go back --------------------------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_rejected_drafts_are_written_over_and_leave_the_scale_of_a_page_that_goes_on(kv):
    """Prompts, drafts of six tokens with much larger values, all but one or none of them taken back: inside a page,
    to a page's border, and from a new page back into the one before."""
    P, n_kv, G = 16, 2, 2
    kept, drafted, left = [5, 16, 29, 12], 6, [6, 16, 30, 16]       # lengths: before, drafted, after the taking back
    made = Made(kv, P, n_kv, G, [40] * 4, 8)
    c, g, want, n = made.c, _gen(9), {"k": {}, "v": {}}, 4
    have = [0] * n

    def append(news, size):
        rows, at, cu = sum(news), 0, [0]
        t = {x: (size * torch.randn(rows, n_kv, 128, generator=g, device=DEV)).to(torch.bfloat16) for x in ("k", "v")}
        for i, m in enumerate(news):
            for x in ("k", "v"):
                if m:
                    _append_oracle(want[x], kv, P, made.rows[i], have[i], t[x][at:at + m].double())
            at += m
            have[i] += m
            cu.append(at)
        c.append(0, K.PagedBatch(_i32(have), made.table, _i32(cu), max(news), rows), t["k"], t["v"])

    def check():
        made.lens = list(have)
        for x in ("k", "v"):
            for i in range(n):
                for j in range(-(-have[i] // P)):
                    for h in range(n_kv):
                        codes, s = want[x][made.rows[i][j], h]
                        held = min(P, have[i] - j * P)
                        assert torch.equal(getattr(c, x + "_pool")[0, made.rows[i][j], h, :held].double(), codes[:held])
                        if kv == "e4m3":
                            assert float(getattr(c, x + "_scale")[0, made.rows[i][j], h]) == s
        for form, m in (("decode", 1), ("few", 3), ("wide", 12)):
            q = torch.randn(n * m, n_kv * G, 128, generator=g, device=DEV).to(torch.bfloat16)
            b = K.PagedBatch(_i32(have), made.table, _i32([m * i for i in range(n + 1)]), m, n * m)
            out, lse = c.decode_attn(0, b, q, lse=True) if form == "decode" else c.prefill_attn(0, b, q, lse=True)
            p_round = 2.0 ** -8 if kv == "bf16" and form == "wide" else 2.0 ** -11
            _check_attention(made, q, out, lse, 128 ** -0.5, [m] * n, True, p_round)

    append(kept, 1.0)
    scales = {} if kv == "bf16" else {x: getattr(c, x + "_scale").clone() for x in ("k", "v")}
    append([drafted] * n, 60.0)
    check()
    have[:] = left
    check()
    if kv == "e4m3":          # the page that holds the last token kept has the scale of the drafts
        page = made.rows[0][0]
        assert all(bool((getattr(c, x + "_scale")[0, page] >= 16 * scales[x][0, page]).all()) for x in ("k", "v"))
    append([1, 3, 3, 1], 1.0)
    check()
    if kv == "e4m3":          # a page begun anew has its own
        for i in (1, 3):
            assert all(bool((getattr(c, x + "_scale")[0, made.rows[i][1]] <= 2.0 ** -6).all()) for x in ("k", "v"))
    assert c.poll_error() == (0, 0)


# ---- making a cache --------------------------------------------------------------------------------------------------

def test_a_cache_made_over_memory_that_queued_work_still_writes_starts_clean():
    """The workspace comes from a block that the current stream has freed while its last write is still queued."""
    cfg = K.make_paged_config(4, 2, 1, 16, 8, 4)
    size = K.paged_sizes(cfg)[2]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        K.PagedKV(cfg, DEV).close()        # its blocks are the allocator's now: what follows makes no new one
        torch.cuda.synchronize()
        old = torch.empty(size, dtype=torch.uint8, device=DEV)
        at = old.data_ptr()
        torch.cuda._sleep(100_000_000)
        old.fill_(1)
        del old
        c = K.PagedKV(cfg, DEV)
        assert c.workspace.data_ptr() == at
        assert not bool(c.workspace[:1024].any())                  # error word and counters
        assert c.poll_error() == (0, 0)


# ---- the largest batch, many heads, captured prompts -----------------------------------------------------------------

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n_kv,G,n", [(1, 4, 256), (1, 8, 33), (48, 1, 5)])
def test_full_batches_with_empty_sequences_and_many_heads(kv, n_kv, G, n):
    """Up to 256 sequences (the most of a call), a third of them without tokens or without new ones; 48 kv heads."""
    P = 16
    lens = [0 if i % 5 == 3 else 1 + (i * 37) % 211 for i in range(n)]
    made = Made(kv, P, n_kv, G, lens, 21)
    c = made.c
    assert c.cfg.max_seqs == n
    for form, top in (("few", 16 // G), ("wide", 23)):
        news = [0 if i % 7 == 2 else 1 + (i * 13) % top for i in range(n)]
        cu = [0]
        for m in news:
            cu.append(cu[-1] + m)
        q = torch.randn(cu[-1], n_kv * G, 128, generator=_gen(top), device=DEV).to(torch.bfloat16)
        out, lse = c.prefill_attn(0, K.PagedBatch(made.kv_len, made.table, _i32(cu), top, cu[-1]), q, lse=True)
        p_round = 2.0 ** -8 if kv == "bf16" and top * G > 16 else 2.0 ** -11
        _check_attention(made, q, out, lse, 128 ** -0.5, news, True, p_round)
    q = torch.randn(n, n_kv * G, 128, generator=_gen(5), device=DEV).to(torch.bfloat16)
    for call in (c.decode_attn, c.prefill_attn):               # prefill without offsets: one token a sequence
        out, lse = call(0, K.PagedBatch(made.kv_len, made.table), q, lse=True)
        _check_attention(made, q, out, lse, 128 ** -0.5, [1] * n, True, 2.0 ** -11)
    # an append over the whole batch: the last tokens of each sequence, stored as they are
    news = [min(t, (i * 29) % 40) for i, t in enumerate(lens)]
    cu = [0]
    for m in news:
        cu.append(cu[-1] + m)
    k, v = (torch.randn(cu[-1], n_kv, 128, generator=_gen(i), device=DEV).to(torch.bfloat16) for i in (1, 2))
    if kv == "e4m3":          # pages that go on: their codes are at most 448, and a large scale stays as it is
        c.k_scale.fill_(1.0)
        c.v_scale.fill_(1.0)
    c.append(0, K.PagedBatch(made.kv_len, made.table, _i32(cu), 39, cu[-1]), k, v)
    assert c.poll_error() == (0, 0)
    for i in range(n):
        for h in range(0, n_kv, 7):
            for got, want in zip(made.held(i, h), (k, v)):
                y = want[cu[i]:cu[i + 1], h].double()
                got = got[lens[i] - news[i]:]
                # half a step of e4m3 under scales of at most 1, or exact
                tol = torch.maximum(2.0 ** -4 * y.abs(), torch.full_like(y, 2.0 ** -10)) if kv == "e4m3" else 0 * y
                assert bool((got - y).abs().le(tol).all()), (i, h)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_captured_prompt_chunks_with_lengths_that_change(kv):
    """append and both kernels of prefill_attn in one graph, replayed with other lengths, offsets and tables; the same
    calls eagerly in between."""
    P, n_kv, G, n, rows = 32, 2, 4, 3, 90
    plans = [([40, 25, 25], [40, 70, 25]), ([1, 80, 0], [41, 150, 25]), ([30, 30, 30], [71, 180, 55]), ([0, 1, 2], [71, 181, 57])]
    ends = plans[-1][1]
    rope = K.Rope(K.rope_table(256, 128), 128)
    toks = {x: torch.randn(len(plans), rows, h, 128, generator=_gen(i), device=DEV).to(torch.bfloat16)
            for i, (x, h) in enumerate((("q", n_kv * G), ("k", n_kv), ("v", n_kv)))}
    results = []
    for mode in ("eager", "captured"):
        made = Made(kv, P, n_kv, G, ends, 4)
        c = made.c
        kv_len, cu, few = _i32([0] * n), _i32([0] * (n + 1)), _i32([0, 2, 4, 6])
        x = {name: torch.zeros_like(t[0]) for name, t in toks.items()}
        b = K.PagedBatch(kv_len, made.table, cu, 80, rows)
        b_few = K.PagedBatch(kv_len, made.table, few, 2, rows)
        qo, out, out_few = (torch.zeros_like(x["q"]) for _ in range(3))

        def step():
            c.append(0, b, x["k"], x["v"], rope=rope, q=x["q"], q_out=qo)
            c.prefill_attn(0, b, qo, out=out)
            c.prefill_attn(0, b_few, qo, out=out_few)

        if mode == "captured":
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        for t, (news, lens) in enumerate(plans):
            kv_len.copy_(_i32(lens))
            cu.copy_(_i32([0, news[0], news[0] + news[1], sum(news)]))
            for name in toks:
                x[name].copy_(toks[name][t])
            out.zero_()
            out_few.zero_()
            graph.replay() if mode == "captured" else step()
            assert c.poll_error() == (0, 0)
            results.append((mode, t, qo.clone(), out.clone(), out_few.clone()))
            if mode == "eager":
                made.lens = lens
                _check_attention(made, qo, out, None, 128 ** -0.5, news, True, 2.0 ** -8 if kv == "bf16" else 2.0 ** -11)
                _check_attention(made, qo, out_few, None, 128 ** -0.5, [2, 2, 2], True, 2.0 ** -11)
                assert not bool(out[sum(news):].any()) and not bool(out_few[6:].any())
    for a, b in zip(results[: len(plans)], results[len(plans):]):
        assert all(torch.equal(p.view(torch.int16), q.view(torch.int16)) for p, q in zip(a[2:], b[2:])), (a[1])
