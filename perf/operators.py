"""The paged KV cache's operators as measured cases: appending keys and values (rotated on the way) to pools held in
bf16 or in e4m3 with a scale for each page and head, attention of single tokens over such a cache, and attention of
several query tokens per sequence (prompt chunks, verification of drafted tokens, cross attention).

A case names the operator, the pool's type and page, the heads, and how the sequences' lengths and new tokens are
spread: n sequences, lengths from lo to hi and new tokens from new_lo to new_hi, both spread over their logarithm.
"""
from __future__ import annotations

import math

import torch

own = False
D = 128
DEV = "cuda"


def _spread(n, lo, hi, shift):
    """n whole numbers from lo to hi, evenly spread over their logarithm in a scattered order (the case alone decides)."""
    if n == 1:
        return [hi]
    at = [((i + 1) * 0.6180339887498949 + shift) % 1.0 for i in range(n)]
    rank = sorted(range(n), key=lambda i: at[i])
    frac = [0.0] * n
    for r, i in enumerate(rank):
        frac[i] = r / (n - 1)
    return [int(round(lo * (hi / lo) ** f)) for f in frac]


def _lens(c):
    """(tokens held, new tokens among them) of each sequence; without a causal mask the two are independent."""
    t = _spread(c["n"], c["lo"], c["hi"], 0.25)
    if c["op"] == "decode":
        return t, [1] * c["n"]
    new = _spread(c["n"], c["new_lo"], c["new_hi"], 0.6)
    if c["op"] == "prefill" and not c["causal"]:
        return t, new
    return [max(a, b) for a, b in zip(t, new)], new


def _case(name, op, kv, page, n_q, n_kv, n, lo, hi, new_lo=1, new_hi=1, causal=True, rot=128, interleaved=False):
    c = dict(op=op, kv=kv, page=page, n_q=n_q, n_kv=n_kv, n=n, lo=lo, hi=hi, new_lo=new_lo, new_hi=new_hi, causal=causal,
             rot=rot, interleaved=interleaved)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # One decode step of 64 sequences: one token each into its open page.
        _case("append-step-64-e4m3", "append", "e4m3", 16, 32, 8, 64, 520, 4100),
        # Ragged prompt chunks of a mixed batch into a bf16 pool, half of the channels rotated in pairs.
        _case("append-ragged-bf16", "append", "bf16", 32, 32, 8, 7, 300, 2500, 3, 1100, rot=64, interleaved=True),
        # A prompt of 32K tokens.
        _case("append-prompt-32k-e4m3", "append", "e4m3", 64, 32, 8, 1, 32768, 32768, 32768, 32768),
        # The smallest decode step, where the launch and the latency count.
        _case("decode-1x4k-e4m3", "decode", "e4m3", 16, 32, 8, 1, 4096, 4096),
        # Four sequences of 32K tokens, not quantised.
        _case("decode-4x32k-bf16", "decode", "bf16", 16, 32, 8, 4, 32768, 32768),
        # A serving batch: 64 sequences of very different lengths.
        _case("decode-mix-64-e4m3", "decode", "e4m3", 32, 32, 8, 64, 700, 32000),
        # One long context, and the longest: few rows, everything in the split over tokens.
        _case("decode-1x128k-e4m3", "decode", "e4m3", 32, 32, 8, 1, 131072, 131072),
        _case("decode-1x1m-e4m3", "decode", "e4m3", 64, 32, 8, 1, 1048576, 1048576),
        # A prompt attended causally as a whole.
        _case("prefill-8k-e4m3", "prefill", "e4m3", 64, 32, 8, 1, 8192, 8192, 8192, 8192),
        # Ragged chunks of a mixed batch behind the contexts already held.
        _case("prefill-ragged-bf16", "prefill", "bf16", 32, 32, 8, 6, 900, 6000, 33, 1500),
        # Verification of five drafted tokens per sequence: few rows against long contexts.
        _case("verify-16x5-e4m3", "prefill", "e4m3", 32, 32, 8, 16, 2000, 16000, 5, 5),
        # Cross attention to an encoder's states, a cache head for each query head.
        _case("cross-8x300-bf16", "prefill", "bf16", 16, 16, 16, 8, 700, 1500, 40, 300, causal=False, rot=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kv, page = rng.choice(["bf16", "e4m3", "e4m3"]), rng.choice([16, 32, 64])
    n_kv = rng.choice([1, 2, 4, 8, 8, 16])
    n_q = n_kv * rng.choice([1, 2, 4, 4, 8])
    op = rng.choice(["append", "decode", "prefill"])
    if op == "append":
        n = _log(rng, 1, 96)
        new_hi = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, 16000 // n))
        hi = _log(rng, max(new_hi, 20), max(new_hi, 20) + 4000)
        return _case(None, op, kv, page, n_q, n_kv, n, _log(rng, 1, hi), hi, _log(rng, 1, new_hi), new_hi,
                     rot=rng.choice([128, 128, 64, 96, 0]), interleaved=rng.random() < 0.3)
    if op == "decode":
        n = _log(rng, 1, 128)
        hi = _log(rng, 50, min(300000, 2000000 // (n * n_kv)))
        return _case(None, op, kv, page, n_q, n_kv, n, _log(rng, max(1, hi // 50), hi), hi)
    n = _log(rng, 1, 24)
    causal = rng.random() < 0.7
    new_hi = _log(rng, 2, max(2, min(4000, 100000 // (n * n_q))))
    hi = _log(rng, max(new_hi, 64), max(new_hi, 64) + 9000 // max(1, n * n_q // 64))
    return _case(None, op, kv, page, n_q, n_kv, n, _log(rng, max(1, hi // 8), hi), hi, _log(rng, 1, new_hi), new_hi,
                 causal=causal, rot=0)


def _pairs(c):
    """Pairs of query token and key that are seen."""
    total = 0
    for t, m in zip(*_lens(c)):
        total += m * t - (m * (m - 1) // 2 if c["causal"] else 0)
    return total


def work(c):
    t, m = _lens(c)
    b = 1 if c["kv"] == "e4m3" else 2
    rows, P = sum(m), c["page"]
    if c["op"] == "append":
        pages = sum((a - 1) // P - (a - k) // P + 1 for a, k in zip(t, m))
        scales = pages * c["n_kv"] * 2 * 4 if b == 1 else 0
        kv = rows * c["n_kv"] * D * 2
        return {"bytes": kv * 2 + kv * b + rows * c["n_q"] * D * 2 * 2 + rows * c["rot"] * 4 + scales,
                "flops": 3 * rows * (c["n_q"] + c["n_kv"]) * c["rot"]}
    held = sum(t) * c["n_kv"] * D * 2 * b
    scales = sum(-(-a // P) for a in t) * c["n_kv"] * 2 * 4 if b == 1 else 0
    return {"bytes": held + scales + rows * c["n_q"] * (D * 2 * 2 + 4),
            "flops": 4 * D * c["n_q"] * (sum(t) if c["op"] == "decode" else _pairs(c))}


def _scale_of(amax):
    """2^e with the smallest whole e >= -64 that holds amax <= 448 * 2^e."""
    m, x = torch.frexp(amax)                      # amax = m 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    e = x - 9 + (m > 0.875).to(x.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, -64)).clamp(min=-64)
    return torch.ldexp(torch.ones_like(amax), e)


def _angles(n, rot):
    """cos and sin of position times base^(-2 i / rot), in 64 bits, rounded once: [n, rot]."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(n, dtype=torch.float64, device=DEV)[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], dim=1).float().contiguous()


def prepare(c, seed):
    t, m = _lens(c)
    P, n, rows = c["page"], c["n"], sum(m)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)

    need = [-(-a // P) for a in t]
    n_pages, cols = sum(need) + 3, max(need)
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(n, cols, dtype=torch.int32, device=DEV)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    # Keys have channels of different sizes; a few are much larger than the rest, as rotated keys have them.
    chan = torch.exp(0.4 * normal(1, c["n_kv"], 1, D))
    chan[..., torch.randperm(D, generator=g, device=DEV)[:3]] *= 4
    s = {"case": c}
    for x, ch in (("k", chan), ("v", torch.exp(0.4 * normal(1, c["n_kv"], 1, D)))):
        pool = torch.empty(1, n_pages, c["n_kv"], P, D, dtype=torch.bfloat16 if c["kv"] == "bf16" else torch.float8_e4m3fn,
                           device=DEV)
        scale = torch.ones(1, n_pages, c["n_kv"], device=DEV)
        step = max(1, (1 << 26) // (c["n_kv"] * P * D))
        for a in range(0, n_pages, step):
            y = normal(min(step, n_pages - a), c["n_kv"], P, D) * ch
            if c["kv"] == "e4m3":
                scale[0, a:a + step] = _scale_of(y.abs().amax(dim=(2, 3)))
                y = y / scale[0, a:a + step, :, None, None]
            pool[0, a:a + step] = y.to(pool.dtype)
        s[x + "_pages"], s[x + "_scale"] = pool, scale if c["kv"] == "e4m3" else None
    s["kv_len"] = torch.tensor(t, dtype=torch.int32, device=DEV)
    ends = [0]
    for k in m:
        ends.append(ends[-1] + k)
    s["cu"] = torch.tensor(ends, dtype=torch.int32, device=DEV)
    s["table"], s["max_new"], s["rows"] = table, max(m), rows
    s["q"] = (1.5 * normal(rows, c["n_q"], D)).to(torch.bfloat16)
    if c["op"] == "append":
        s["k"] = (normal(rows, c["n_kv"], D) * chan[:, :, 0]).to(torch.bfloat16)
        s["v"] = normal(rows, c["n_kv"], D).to(torch.bfloat16)
        s["angles"] = _angles(max(t), c["rot"]) if c["rot"] else None
        s["q_out"] = torch.empty_like(s["q"])
    else:
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(rows, c["n_q"], dtype=torch.float32, device=DEV)
    if own:
        from compressed_kv_cache_vector_gb300 import binding as B
        cfg = B.make_paged_config(c["n_q"], c["n_kv"], 1, P, n_pages, n, B.MK_KV_E4M3 if c["kv"] == "e4m3" else B.MK_KV_BF16)
        s["cache"] = B.PagedKV(cfg, DEV, s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
        step = c["op"] == "decode" or s["max_new"] == 1
        s["batch"] = B.PagedBatch(s["kv_len"], table, None if step else s["cu"], s["max_new"], rows)
        s["rope"] = B.Rope(s["angles"], c["rot"], c["interleaved"]) if s.get("angles") is not None else None
    return s


# ---- the plain forms -------------------------------------------------------------------------------------------------

def _where(s):
    """Of each new token: its sequence, its position there, its page and its slot."""
    cu, kv_len, P = s["cu"].long(), s["kv_len"].long(), s["case"]["page"]
    row = torch.arange(s["rows"], device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    pos = kv_len[seq] - (cu[seq + 1] - cu[seq]) + row - cu[seq]
    return seq, pos, s["table"][seq, pos // P].long(), pos % P


def _rotated(x, angles, pos, rot, interleaved):
    y = x.float()
    if not rot:
        return y
    h = rot // 2
    c, sn = angles[pos][:, None, :h], angles[pos][:, None, h:]
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :h], y[..., h:rot])
    p, r = a * c - b * sn, b * c + a * sn
    z = y.clone()
    if interleaved:
        z[..., 0:rot:2], z[..., 1:rot:2] = p, r
    else:
        z[..., :h], z[..., h:rot] = p, r
    return z


def _plain_append(s):
    c = s["case"]
    P = c["page"]
    seq, pos, page, slot = _where(s)
    s["q_out"].copy_(_rotated(s["q"], s["angles"], pos, c["rot"], c["interleaved"]))
    head = torch.arange(c["n_kv"], device=DEV)
    new = s["cu"][1:].long() - s["cu"][:-1].long()
    old = s["kv_len"].long() - new
    first = s["table"].gather(1, (old // P).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long()
    for x, y in (("k", _rotated(s["k"], s["angles"], pos, c["rot"], c["interleaved"])), ("v", s["v"].float())):
        pool, scale = s[x + "_pages"][0], s[x + "_scale"]
        if c["kv"] == "bf16":
            pool[page[:, None], head[None, :], slot[:, None]] = y.to(torch.bfloat16)
            continue
        scale = scale[0]
        top = torch.zeros_like(scale).index_reduce_(0, page, y.abs().amax(dim=2), "amax")
        was = scale.clone()
        fresh = torch.zeros(scale.shape[0], device=DEV).index_add_(0, page, (slot == 0).float())[:, None] > 0
        hit = torch.zeros(scale.shape[0], device=DEV).index_add_(0, page, torch.ones_like(slot, dtype=torch.float32))[:, None] > 0
        now = torch.where(hit, torch.maximum(torch.where(fresh, torch.zeros_like(was), was), _scale_of(top)), was)
        scale.copy_(now)
        # Tokens held before in a page that gets new ones are brought to its new scale.
        ratio = (was / now)[first]
        held = pool.view(torch.uint8)[first].view(torch.float8_e4m3fn)
        again = (held.float() * ratio[:, :, None, None]).to(torch.float8_e4m3fn)
        keep = (torch.arange(P, device=DEV)[None, :] < (old % P)[:, None])[:, None, :, None] & (new > 0)[:, None, None, None]
        pool.view(torch.uint8)[first] = torch.where(keep, again.view(torch.uint8), held.view(torch.uint8))
        code = (y / now[page][:, :, None]).to(torch.float8_e4m3fn)
        pool.view(torch.uint8)[page[:, None], head[None, :], slot[:, None]] = code.view(torch.uint8)


def _held(s, x):
    """The cache's values of every sequence, padded to the longest: [n, heads, tokens, 128] in 32 bits."""
    t = s["table"].long()
    y = s[x + "_pages"][0].view(torch.uint8)[t].view(s[x + "_pages"].dtype).float()      # [n, pages, heads, P, 128]
    if s[x + "_scale"] is not None:
        y = y * s[x + "_scale"][0][t][..., None, None]
    n, k, h, P, d = y.shape
    return y.transpose(1, 2).reshape(n, h, k * P, d)


def _plain_attention(s):
    c = s["case"]
    n, G, H = c["n"], c["n_q"] // c["n_kv"], c["n_kv"]
    K = _held(s, "k")
    T, M = K.shape[2], s["max_new"]
    cu, kv_len = s["cu"].long(), s["kv_len"].long()
    new = cu[1:] - cu[:-1]
    at = torch.arange(M, device=DEV)
    row = (cu[:-1, None] + at[None, :]).clamp(max=s["rows"] - 1)                          # [n, M]
    q = s["q"][row].float().view(n, M, H, G, D).permute(0, 2, 3, 1, 4).reshape(n, H, G * M, D)
    sees = kv_len[:, None].expand(n, M)
    if c["causal"]:
        sees = sees - new[:, None] + at[None, :] + 1
    hid = (torch.arange(T, device=DEV)[None, None, :] >= sees[:, :, None])[:, None, None]  # [n, 1, 1, M, T]
    z = torch.matmul(q, K.transpose(2, 3)).mul_(1 / math.sqrt(D)).view(n, H, G, M, T)
    del K
    z.masked_fill_(hid, -math.inf)
    top = z.amax(dim=4, keepdim=True)
    z = z.sub_(top).exp_()
    total = z.sum(dim=4, keepdim=True)
    o = torch.matmul(z.view(n, H, G * M, T), _held(s, "v")).view(n, H, G, M, D) / total
    real = at[None, :] < new[:, None]
    o = o.permute(0, 3, 1, 2, 4).reshape(n, M, c["n_q"], D)
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(n, M, c["n_q"])
    flat = torch.where(real, row, torch.full_like(row, s["rows"])).reshape(-1)
    out = torch.zeros(s["rows"] + 1, c["n_q"], D, device=DEV).index_copy_(0, flat, o.reshape(n * M, c["n_q"], D))
    ls = torch.zeros(s["rows"] + 1, c["n_q"], device=DEV).index_copy_(0, flat, lse.reshape(n * M, c["n_q"]))
    s["out"].copy_(out[:-1])
    s["lse"].copy_(ls[:-1])


def run(s):
    c = s["case"]
    if c["op"] == "append":
        if own:
            s["cache"].append(0, s["batch"], s["k"], s["v"], rope=s["rope"], q=s["q"], q_out=s["q_out"])
        else:
            _plain_append(s)
        return {"k": s["k_pages"], "v": s["v_pages"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "q": s["q_out"]}
    if not own:
        _plain_attention(s)
    elif c["op"] == "decode":
        s["cache"].decode_attn(0, s["batch"], s["q"], out=s["out"], lse=s["lse"])
    else:
        s["cache"].prefill_attn(0, s["batch"], s["q"], causal=c["causal"], out=s["out"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------

def _e4m3(x):
    """Nearest value of 4 exponent and 3 mantissa bits, ties to even, at most 448, of doubles."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(c, s):
    t, m = _lens(c)
    P, H, h = c["page"], c["n_kv"], c["rot"] // 2
    res = {x: s[x].double() for x in ("k_pages", "v_pages")}
    sc = {x: s[x + "_scale"].double() if s[x + "_scale"] is not None else None for x in ("k", "v")}
    table = s["table"].tolist()
    q_out, at = torch.empty(s["rows"], c["n_q"], D, dtype=torch.float64, device=DEV), 0

    def turn(x, first):
        z = x.double().clone()
        if h:
            a = s["angles"][first:first + x.shape[0]].double()[:, None]
            i = torch.arange(h, device=DEV)
            p, r = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + h)
            w = torch.complex(z[..., p], z[..., r]) * torch.complex(a[..., :h], a[..., h:])
            z[..., p], z[..., r] = w.real, w.imag
        return z

    for i, (length, new) in enumerate(zip(t, m)):
        start = length - new
        q_out[at:at + new] = turn(s["q"][at:at + new], start)
        rows = {"k": turn(s["k"][at:at + new], start), "v": s["v"][at:at + new].double()}
        for j in range(start // P, -(-length // P)):
            a, b, page = max(start, j * P), min(length, (j + 1) * P), table[i][j]
            for x in ("k", "v"):
                y = rows[x][a - start:b - start].transpose(0, 1)                # [heads, tokens, 128]
                pool = res[x + "_pages"][0, page]
                if c["kv"] == "bf16":
                    pool[:, a - j * P:b - j * P] = y
                    continue
                top = y.abs().amax(dim=(1, 2))
                e = torch.ceil(torch.log2(top / 448)).clamp(min=-64)
                one = torch.exp2(e)
                if a > j * P:
                    was = sc[x][0, page]
                    one = torch.maximum(one, was)
                    pool[:, :a - j * P] = _e4m3(pool[:, :a - j * P] * (was / one)[:, None, None])
                pool[:, a - j * P:b - j * P] = _e4m3(y / one[:, None, None])
                sc[x][0, page] = one
        at += new
    return {"k": res["k_pages"], "v": res["v_pages"], "k_scale": sc["k"], "v_scale": sc["v"], "q": q_out}


def _exact_attention(c, s):
    t, m = _lens(c)
    P, G = c["page"], c["n_q"] // c["n_kv"]
    out = torch.zeros(s["rows"], c["n_q"], D, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["rows"], c["n_q"], dtype=torch.float64, device=DEV)
    at = 0
    for i, (length, new) in enumerate(zip(t, m)):
        pages = s["table"][i, : -(-length // P)].long()
        for h in range(c["n_kv"]):
            k, v = (s[x + "_pages"][0, :, h].view(torch.uint8)[pages].view(s[x + "_pages"].dtype).double() for x in ("k", "v"))
            if s["k_scale"] is not None:
                k = k * s["k_scale"][0, pages, h].double()[:, None, None]
                v = v * s["v_scale"][0, pages, h].double()[:, None, None]
            k, v = k.reshape(-1, D)[:length], v.reshape(-1, D)[:length]
            for a in range(0, new, 2048):
                b = min(new, a + 2048)
                q = s["q"][at + a:at + b, h * G:(h + 1) * G].double()
                z = torch.einsum("mgd,td->mgt", q, k) / math.sqrt(D)
                if c["causal"]:
                    last = length - new + torch.arange(a, b, device=DEV)
                    z = z.masked_fill((torch.arange(length, device=DEV)[None, :] > last[:, None])[:, None], -math.inf)
                lse[at + a:at + b, h * G:(h + 1) * G] = torch.logsumexp(z, dim=2)
                out[at + a:at + b, h * G:(h + 1) * G] = torch.einsum("mgt,td->mgd", torch.softmax(z, dim=2), v)
        at += new
    return {"out": out, "lse": lse}


def exact(c, seed):
    s = prepare(c, seed)
    return _exact_append(c, s) if c["op"] == "append" else _exact_attention(c, s)
