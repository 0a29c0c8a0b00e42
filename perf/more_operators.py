"""More operators of the paged KV cache as measured cases: attention of single tokens for sequences that share a long
prefix (its pages are read once for all of them), the attention mass of every held token (the softmax weights that it
got, summed over queries and over the query heads of its kv head) with a decode step or for a prompt's queries, and
eviction: a sequence keeps its first, its last and its heaviest tokens, moved together to the front of its pages.

A case names the operator, the pool's type and page, the heads, and how lengths are spread over n sequences.
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


def _prefix(name, kv, page, n_kv, g, n, groups, lo, hi, tail_lo, tail_hi):
    """n sequences in `groups` groups; a group shares lo to hi tokens, a sequence has tail_lo to tail_hi of its own."""
    return _named(name, dict(op="prefix", kv=kv, page=page, n_kv=n_kv, n_q=n_kv * g, n=n, groups=groups, lo=lo, hi=hi,
                             tail_lo=tail_lo, tail_hi=tail_hi))


def _step(name, kv, page, n_kv, g, n, lo, hi):
    """A decode step of n sequences of lo to hi tokens that also adds to the tokens' mass."""
    return _named(name, dict(op="step", kv=kv, page=page, n_kv=n_kv, n_q=n_kv * g, n=n, lo=lo, hi=hi))


def _prompt(name, kv, page, n_kv, g, n, lo, hi, new_lo, new_hi, add):
    """The mass that the last new_lo to new_hi tokens' queries give to the lo to hi held tokens of n sequences; add: to
    the mass that the tokens before them have, else it begins anew."""
    return _named(name, dict(op="prompt", kv=kv, page=page, n_kv=n_kv, n_q=n_kv * g, n=n, lo=lo, hi=hi, new_lo=new_lo,
                             new_hi=new_hi, add=add))


def _evict(name, kv, page, n_kv, n, lo, hi, share, first, recent):
    """n sequences of lo to hi tokens keep about `share` of them, among these the first and the recent ones."""
    return _named(name, dict(op="evict", kv=kv, page=page, n_kv=n_kv, n_q=n_kv * 4, n=n, lo=lo, hi=hi, share=share,
                             first=first, recent=recent))


def _named(name, c):
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # Eight conversations behind a system prompt of 2K tokens.
        _prefix("prefix-8-on-2k-e4m3", "e4m3", 16, 8, 4, 8, 1, 2048, 2048, 20, 300),
        # Many answers to one question about a document: 32 samples, a 64K document, not quantised.
        _prefix("prefix-32-on-64k-bf16", "bf16", 32, 8, 4, 32, 1, 65536, 65536, 40, 600),
        # A serving batch whose sequences share several prompts of different lengths.
        _prefix("prefix-96-on-7-e4m3", "e4m3", 32, 8, 4, 96, 7, 900, 20000, 15, 1800),
        # A large batch of samples from one long prompt.
        _prefix("prefix-192-on-32k-e4m3", "e4m3", 64, 8, 4, 192, 1, 32500, 32500, 30, 900),
        # The smallest decode step with mass, where launches and latency count.
        _step("step-1x4k-e4m3", "e4m3", 16, 8, 4, 1, 4100, 4100),
        # A serving batch of different lengths.
        _step("step-mix-48-e4m3", "e4m3", 32, 8, 4, 48, 500, 20000),
        # Long contexts, not quantised.
        _step("step-3x100k-bf16", "bf16", 64, 8, 4, 3, 90000, 110000),
        # A whole prompt: every query counts for every token before it.
        _prompt("prompt-6k-e4m3", "e4m3", 32, 8, 4, 1, 6000, 6000, 6000, 6000, False),
        # Ragged chunks behind what is held already.
        _prompt("prompt-chunks-5-bf16", "bf16", 16, 8, 4, 5, 1500, 9000, 60, 1300, True),
        # A window of the last queries of long prompts decides what is kept.
        _prompt("prompt-window-6x32-e4m3", "e4m3", 64, 8, 4, 6, 5000, 40000, 32, 32, False),
        # One long context cut to a quarter.
        _evict("evict-1x64k-e4m3", "e4m3", 32, 8, 1, 65536, 65536, 0.25, 4, 256),
        # A batch of different lengths cut to about half.
        _evict("evict-24-bf16", "bf16", 16, 8, 24, 700, 9000, 0.5, 4, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kv, page = rng.choice(["bf16", "e4m3", "e4m3"]), rng.choice([16, 32, 64])
    n_kv, g = rng.choice([1, 2, 4, 8, 8, 16]), rng.choice([1, 2, 4, 4, 8])
    op = rng.choice(["prefix", "step", "prompt", "evict"])
    if op == "prefix":
        n = _log(rng, 2, 200)
        groups = 1 if rng.random() < 0.5 else rng.randint(1, max(1, n // 3))
        hi = _log(rng, 100, max(200, min(100000, 150000000 // (n * n_kv * g), 1000000 // (groups * n_kv))))
        tail_hi = _log(rng, 2, max(3, min(4000, 300000 // (n * n_kv) * 4)))
        return _prefix(None, kv, page, n_kv, g, n, groups, _log(rng, max(1, hi // 20), hi), hi, _log(rng, 1, tail_hi), tail_hi)
    if op == "step":
        n = _log(rng, 1, 100)
        hi = _log(rng, 50, min(200000, 1500000 // (n * n_kv)))
        return _step(None, kv, page, n_kv, g, n, _log(rng, max(1, hi // 50), hi), hi)
    if op == "prompt":
        n = _log(rng, 1, 20)
        new_hi = _log(rng, 2, max(3, min(5000, 150000 // (n * n_kv * g))))
        hi = _log(rng, max(new_hi, 64), max(new_hi, 64) + min(100000, 200000000 // (n * n_kv * g * new_hi), 1000000 // (n * n_kv)))
        return _prompt(None, kv, page, n_kv, g, n, _log(rng, max(1, hi // 8), hi), hi, _log(rng, 1, new_hi), new_hi, rng.random() < 0.5)
    n = _log(rng, 1, 64)
    hi = _log(rng, 60, min(120000, 700000 // (n * n_kv)))
    return _evict(None, kv, page, n_kv, n, _log(rng, max(1, hi // 20), hi), hi, rng.choice([0.1, 0.25, 0.5, 0.8]),
                  rng.choice([0, 4, 70]), rng.choice([0, 16, 100]))


def _lens(c):
    """Tokens held by each sequence, new tokens among them, and for each group its sequences and what they share."""
    n = c["n"]
    if c["op"] != "prefix":
        t = _spread(n, c["lo"], c["hi"], 0.25)
        new = _spread(n, c["new_lo"], c["new_hi"], 0.6) if c["op"] == "prompt" else [1] * n
        return [max(a, b) for a, b in zip(t, new)], new, [], []
    size = _spread(c["groups"], 1, 4, 0.1)
    ends = [round(n * sum(size[:i]) / sum(size)) for i in range(len(size) + 1)]
    shared, tails = _spread(c["groups"], c["lo"], c["hi"], 0.4), _spread(n, c["tail_lo"], c["tail_hi"], 0.25)
    return [tails[i] + shared[g] for g in range(len(size)) for i in range(ends[g], ends[g + 1])], [1] * n, ends, shared


def _kept(c):
    """Tokens that each sequence keeps."""
    return [min(t, max(c["first"] + c["recent"], int(t * c["share"]))) for t in _lens(c)[0]]


def work(c):
    t, m, ends, shared = _lens(c)
    b = 1 if c["kv"] == "e4m3" else 2
    P, H, nq, rows = c["page"], c["n_kv"], c["n_q"], sum(m)
    scales = lambda tokens: -(-tokens // P) * H * 2 * 4 if b == 1 else 0  # noqa: E731
    if c["op"] == "evict":
        k = [y for x, y in zip(t, _kept(c)) if y < x]
        data = 2 * sum(k) * H * D * 2 * b                                   # keys and values read and written
        return {"bytes": data + sum(scales(x) + scales(y) for x, y in zip(t, _kept(c)) if y < x)
                + 4 * H * (sum(x for x, y in zip(t, _kept(c)) if y < x) + 3 * sum(k)), "flops": 0}
    if c["op"] == "prefix":
        own_t = [x - s // P * P for g, s in enumerate(shared) for x in t[ends[g]:ends[g + 1]]]
        once = [s // P * P for g, s in enumerate(shared) if ends[g + 1] > ends[g]]
        return {"bytes": sum(x * H * D * 2 * b + scales(x) for x in own_t + once) + rows * nq * (D * 2 * 2 + 4),
                "flops": 4 * D * nq * sum(t)}
    if c["op"] == "step":
        return {"bytes": sum(x * H * (D * 2 * b + 8) + scales(x) for x in t) + rows * nq * (D * 2 * 2 + 4), "flops": 4 * D * nq * sum(t)}
    pairs = sum(k * x - k * (k - 1) // 2 for x, k in zip(t, m))
    return {"bytes": sum(x * H * (D * b + (8 if c["add"] else 4)) + scales(x) // 2 for x in t) + rows * nq * (D * 2 + 4), "flops": 2 * D * nq * pairs}


def _scale_of(amax):
    """2^e with the smallest whole e >= -64 that holds amax <= 448 * 2^e."""
    m, x = torch.frexp(amax)                      # amax = m 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    e = x - 9 + (m > 0.875).to(x.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, -64)).clamp(min=-64)
    return torch.ldexp(torch.ones_like(amax), e)


def prepare(c, seed):
    t, m, ends, shared = _lens(c)
    P, n, rows = c["page"], c["n"], sum(m)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    # Pages in scattered order; sequences of a group name the same ones for the whole pages that they share.
    common = [0] * n
    for j in range(len(shared)):
        common[ends[j]:ends[j + 1]] = [shared[j] // P] * (ends[j + 1] - ends[j])
    need = [-(-a // P) - k for a, k in zip(t, common)]
    n_pages = sum(need) + sum(s // P for s in shared) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(n, max(-(-a // P) for a in t), dtype=torch.int32, device=DEV)
    at = 0
    for j in range(len(shared)):
        table[ends[j]:ends[j + 1], :shared[j] // P] = order[at:at + shared[j] // P]
        at += shared[j] // P
    for i in range(n):
        table[i, common[i]:common[i] + need[i]] = order[at:at + need[i]]
        at += need[i]
    # Keys have channels of different sizes; a few are much larger than the rest, as rotated keys have them.
    chan = torch.exp(0.4 * normal(1, c["n_kv"], 1, D))
    chan[..., torch.randperm(D, generator=g, device=DEV)[:3]] *= 4
    s = {"case": c, "table": table}
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
    if c["op"] == "evict":
        # Mass as prompts leave it: a few heavy tokens, many light ones, some that no query ever looked at.
        w = torch.exp(2 * normal(1, n_pages, c["n_kv"], P))
        s["mass"] = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.05, torch.zeros_like(w), w)
        s["keep"] = torch.tensor(_kept(c), dtype=torch.int32, device=DEV)
        s["kept"] = torch.zeros(n, c["n_kv"], max(_kept(c)), dtype=torch.int32, device=DEV)
        s["new_len"] = torch.zeros(n, dtype=torch.int32, device=DEV)
    else:
        cu = [0]
        for k in m:
            cu.append(cu[-1] + k)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["max_new"], s["rows"] = max(m), rows
        s["q"] = (1.5 * normal(rows, c["n_q"], D)).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(rows, c["n_q"], device=DEV)
        if c["op"] in ("step", "prompt"):
            s["mass"] = torch.exp(normal(1, n_pages, c["n_kv"], P))
        if c["op"] == "prompt":  # the prompt's attention has left the logarithms of the rows' sums
            at = 0
            for i in range(n):
                pages = table[i, : -(-t[i] // P)].long()
                k = s["k_pages"][0].view(torch.uint8)[pages].view(s["k_pages"].dtype).float()
                k = k * s["k_scale"][0, pages][..., None, None] if s["k_scale"] is not None else k
                k = k.transpose(0, 1).reshape(c["n_kv"], -1, D)[:, :t[i]]
                for a in range(0, m[i], 1024):
                    b = min(m[i], a + 1024)
                    q = s["q"][at + a:at + b].float().view(b - a, c["n_kv"], -1, D)
                    z = torch.einsum("mhgd,htd->mhgt", q, k) * D ** -0.5
                    hid = torch.arange(t[i], device=DEV) > (t[i] - m[i] + torch.arange(a, b, device=DEV))[:, None]
                    z = z.masked_fill(hid[:, None, None], -math.inf)
                    s["lse"][at + a:at + b] = torch.logsumexp(z, dim=3).reshape(b - a, -1)
                at += m[i]
        if c["op"] == "prefix":
            s["cu_group"] = torch.tensor(ends, dtype=torch.int32, device=DEV)
            s["prefix_len"] = torch.tensor(shared, dtype=torch.int32, device=DEV)
            s["most"] = max(b - a for a, b in zip(ends, ends[1:])), max(a // P for a in shared)
            s["most_own"] = max(need)
    if own:
        from compressed_kv_cache_vector_gb300 import binding as B
        cfg = B.make_paged_config(c["n_q"], c["n_kv"], 1, P, n_pages, n, B.MK_KV_E4M3 if c["kv"] == "e4m3" else B.MK_KV_BF16)
        s["cache"] = B.PagedKV(cfg, DEV, s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
        if c["op"] == "prompt":
            s["batch"] = B.PagedBatch(s["kv_len"], table, s["cu"], s["max_new"], rows)
        else:
            s["batch"] = B.PagedBatch(s["kv_len"], table)
        if "mass" in s:
            s["own_mass"] = B.PagedMass(s["cache"], s["mass"])
        if c["op"] == "prefix":
            s["prefix"] = B.PagedPrefix(s["cu_group"], s["prefix_len"])
    return s


# ---- the plain forms -------------------------------------------------------------------------------------------------

def _values(s, x, table):
    """What the pages of a table [n, columns] hold: [n, heads, columns * page, 128] in 32 bits."""
    t = table.long()
    y = s[x + "_pages"][0].view(torch.uint8)[t].view(s[x + "_pages"].dtype).float()      # [n, pages, heads, P, 128]
    if s[x + "_scale"] is not None:
        y = y * s[x + "_scale"][0][t][..., None, None]
    n, k, h, P, d = y.shape
    return y.transpose(1, 2).reshape(n, h, k * P, d)


def _part(q, k, v, hid):
    """Maximum, sum and weighted values of rows q [n, heads, m, 128] over keys that are not hidden."""
    z = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).masked_fill_(hid, -math.inf)
    top = z.amax(dim=3, keepdim=True).clamp_(min=-1e30)
    z = z.sub_(top).exp_()
    return top, z.sum(dim=3, keepdim=True), torch.matmul(z, v)


def _plain_prefix(s):
    c = s["case"]
    P, H, n, G = c["page"], c["n_kv"], c["n"], c["n_q"] // c["n_kv"]
    members, columns = s["most"]
    cu, whole = s["cu_group"].long(), s["prefix_len"].long() // P
    seq = torch.arange(n, device=DEV)
    group = torch.searchsorted(cu[1:].contiguous(), seq, right=True)
    q = s["q"].float().view(n, H, G, D)
    # A group's rows against what it shares, padded to the largest group and the longest prefix.
    at = (cu[:-1, None] + torch.arange(members, device=DEV)).clamp(max=n - 1)
    rows = q[at].permute(0, 2, 1, 3, 4).reshape(len(cu) - 1, H, members * G, D)
    table = s["table"][cu[:-1].clamp(max=n - 1), :max(1, columns)]
    hid = torch.arange(max(1, columns) * P, device=DEV)[None, :] >= whole[:, None] * P
    parts = _part(rows, _values(s, "k", table), _values(s, "v", table), hid[:, None, None])
    place = (seq - cu[group])
    top, total, o = (x.view(len(cu) - 1, H, members, G, -1)[group, :, place] for x in parts)
    # Every sequence's own tokens.
    column = (whole[group][:, None] + torch.arange(s["most_own"], device=DEV)).clamp(max=s["table"].shape[1] - 1)
    table = s["table"].gather(1, column)
    left = s["kv_len"].long() - whole[group] * P
    hid = torch.arange(s["most_own"] * P, device=DEV)[None, :] >= left[:, None]
    top2, total2, o2 = _part(q, _values(s, "k", table), _values(s, "v", table), hid[:, None, None])
    most = torch.maximum(top, top2)
    a, b = torch.exp(top - most), torch.exp(top2 - most)
    sums = total * a + total2 * b
    s["out"].copy_(((o * a + o2 * b) / sums).reshape(n, c["n_q"], D))
    s["lse"].copy_((most + sums.log()).reshape(n, c["n_q"]))


def _add_mass(s, w, begins):
    """Adds w [n, heads, tokens] to the held tokens' mass; from token begins[i] on (and with no addition at all: from 0)
    it is the mass."""
    P, n, T = s["case"]["page"], w.shape[0], w.shape[2]
    token = torch.arange(T, device=DEV)
    seq, tok = (token[None, :] < s["kv_len"][:, None]).nonzero(as_tuple=True)
    page, slot = s["table"][seq, tok // P].long(), tok % P
    mass, head = s["mass"][0], torch.arange(w.shape[1], device=DEV)
    old = mass[page[:, None], head[None, :], slot[:, None]]
    old = torch.where((tok >= begins[seq])[:, None], torch.zeros_like(old), old)
    mass[page[:, None], head[None, :], slot[:, None]] = old + w[seq, :, tok]


def _plain_step(s):
    c = s["case"]
    n, H, G = c["n"], c["n_kv"], c["n_q"] // c["n_kv"]
    q = s["q"].float().view(n, H, G, D)
    k = _values(s, "k", s["table"])
    hid = (torch.arange(k.shape[2], device=DEV)[None, :] >= s["kv_len"][:, None])[:, None, None]
    z = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).masked_fill_(hid, -math.inf)
    del k
    top = z.amax(dim=3, keepdim=True)
    z = z.sub_(top).exp_()
    total = z.sum(dim=3, keepdim=True)
    s["lse"].copy_((top + total.log()).reshape(n, c["n_q"]))
    z = z.div_(total)
    s["out"].copy_(torch.matmul(z, _values(s, "v", s["table"])).reshape(n, c["n_q"], D))
    _add_mass(s, z.sum(dim=2), s["kv_len"].long() - 1)


def _plain_prompt(s):
    c = s["case"]
    n, H, G, M = c["n"], c["n_kv"], c["n_q"] // c["n_kv"], s["max_new"]
    k = _values(s, "k", s["table"])
    T = k.shape[2]
    cu, kv_len = s["cu"].long(), s["kv_len"].long()
    new = cu[1:] - cu[:-1]
    at = torch.arange(M, device=DEV)
    row = (cu[:-1, None] + at[None, :]).clamp(max=s["rows"] - 1)                          # [n, M]
    q = s["q"][row].float().view(n, M, H, G, D).permute(0, 2, 3, 1, 4).reshape(n, H, G * M, D)
    lse = s["lse"][row].view(n, M, H, G).permute(0, 2, 3, 1)                              # [n, H, G, M]
    sees = kv_len[:, None] - new[:, None] + at[None, :] + 1
    hid = (torch.arange(T, device=DEV)[None, None, :] >= sees[:, :, None]) | (at[None, :] >= new[:, None])[:, :, None]
    z = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).view(n, H, G, M, T)
    z = z.sub_(lse[..., None]).exp_().masked_fill_(hid[:, None, None], 0)
    _add_mass(s, z.sum(dim=(2, 3)), kv_len - new if c["add"] else torch.zeros_like(new))


def _plain_evict(s):
    c = s["case"]
    P, n, H = c["page"], c["n"], c["n_kv"]
    kv_len, keep, table = s["kv_len"].long(), s["keep"].long(), s["table"].long()
    T, K = table.shape[1] * P, s["kept"].shape[2]
    token = torch.arange(T, device=DEV)
    held = s["mass"][0][table].transpose(1, 2).reshape(n, H, T)
    always = (token[None, :] < c["first"]) | (token[None, :] >= kv_len[:, None] - c["recent"])
    rank = torch.where(always[:, None], torch.full_like(held, math.inf), held)
    rank = torch.where((token[None, :] < kv_len[:, None])[:, None], rank, torch.full_like(held, -math.inf))
    order = rank.sort(dim=2, descending=True, stable=True).indices[..., :K]               # ties: the lowest token first
    stay = torch.arange(K, device=DEV)[None, :] < torch.minimum(keep, kv_len)[:, None]
    kept = torch.where(stay[:, None], order, torch.full_like(order, T)).sort(dim=2).values
    kept = torch.where(stay[:, None], kept, torch.zeros_like(kept))                       # [n, H, K] ascending
    s["kept"].copy_(torch.where(stay[:, None], kept, s["kept"].long()))
    s["new_len"].copy_(torch.minimum(keep, kv_len))
    head = torch.arange(H, device=DEV)[None, :, None]
    slots = -(-K // P) * P
    pad = torch.nn.functional.pad(kept, (0, slots - K))
    real = torch.nn.functional.pad(stay, (0, slots - K))[:, None].expand(n, H, slots)
    moved = (pad != torch.arange(slots, device=DEV)) & real
    page = table.gather(1, pad.view(n, -1) // P).view(n, H, slots)
    to = table[:, :slots // P]
    new_mass = s["mass"][0][page, head, pad % P]
    hit = moved.view(n, H, slots // P, P).any(dim=3)                                      # pages with a token from elsewhere
    seq, h, j = hit.nonzero(as_tuple=True)
    where = real.view(n, H, slots // P, P)[seq, h, j]
    dst = to[seq, j]
    s["mass"][0][dst, h] = torch.where(where, new_mass.view(n, H, slots // P, P)[seq, h, j], s["mass"][0][dst, h])
    new = {}
    for x in ("k", "v"):
        pool = s[x + "_pages"][0]
        raw = pool.view(torch.uint8).view(pool.shape[:3] + (-1,))
        p, o = page.view(n, H, -1, P)[seq, h, j], pad.view(n, H, -1, P)[seq, h, j] % P
        y = raw[p, h[:, None], o].view(pool.dtype)
        if c["kv"] == "e4m3":
            y = y.float() * s[x + "_scale"][0][p, h[:, None]][..., None]
            sc = _scale_of((y.abs() * where[..., None]).amax(dim=(1, 2)))
            new[x + "s"], y = sc, (y / sc[:, None, None]).to(torch.float8_e4m3fn)
        new[x] = torch.where(where[..., None], y.view(torch.uint8), raw[dst, h])
    for x in ("k", "v"):
        pool = s[x + "_pages"][0]
        pool.view(torch.uint8).view(pool.shape[:3] + (-1,))[dst, h] = new[x]
        if c["kv"] == "e4m3":
            s[x + "_scale"][0][dst, h] = new[x + "s"]


def run(s):
    c = s["case"]
    if c["op"] == "evict":
        if own:
            s["cache"].evict(0, s["batch"], s["own_mass"], s["keep"], first=c["first"], recent=c["recent"], kept=s["kept"],
                             new_len=s["new_len"])
        else:
            _plain_evict(s)
        return {"k": s["k_pages"], "v": s["v_pages"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "mass": s["mass"],
                "kept": s["kept"], "new_len": s["new_len"]}
    if c["op"] == "prompt":
        if own:
            s["cache"].prefill_mass(0, s["batch"], s["q"], s["lse"], s["own_mass"], add=c["add"])
        else:
            _plain_prompt(s)
        return {"mass": s["mass"]}
    if c["op"] == "step":
        if own:
            s["cache"].decode_attn_mass(0, s["batch"], s["q"], s["own_mass"], out=s["out"], lse=s["lse"])
        else:
            _plain_step(s)
        return {"out": s["out"], "lse": s["lse"], "mass": s["mass"]}
    if own:
        s["cache"].prefix_attn(0, s["batch"], s["prefix"], s["q"], out=s["out"], lse=s["lse"])
    else:
        _plain_prefix(s)
    return {"out": s["out"], "lse": s["lse"]}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------

def _e4m3(x):
    """Nearest value of 4 exponent and 3 mantissa bits, ties to even, at most 448, of doubles."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_rows(s, x, i, length):
    """One sequence's values [heads, length, 128] as doubles."""
    P = s["case"]["page"]
    pages = s["table"][i, : -(-length // P)].long()
    y = s[x + "_pages"][0].view(torch.uint8)[pages].view(s[x + "_pages"].dtype).double()
    if s[x + "_scale"] is not None:
        y = y * s[x + "_scale"][0, pages].double()[..., None, None]
    return y.transpose(0, 1).reshape(y.shape[1], -1, D)[:, :length]


def _exact_mass(s, i, length):
    P = s["case"]["page"]
    pages = s["table"][i, : -(-length // P)].long()
    return pages, s["mass"][0, pages].double().transpose(0, 1).reshape(s["case"]["n_kv"], -1)[:, :length]


def _put_mass(res, s, pages, w):
    P, (h, T) = s["case"]["page"], w.shape
    tok = torch.arange(T, device=DEV)
    res[0, pages[tok // P][:, None], torch.arange(h, device=DEV), (tok % P)[:, None]] = w.T


def _exact_attention(c, s):
    """prefix and step: every sequence by itself over all that it holds."""
    t, _, ends, shared = _lens(c)
    G = c["n_q"] // c["n_kv"]
    out = torch.empty(c["n"], c["n_q"], D, dtype=torch.float64, device=DEV)
    lse = torch.empty(c["n"], c["n_q"], dtype=torch.float64, device=DEV)
    res = s["mass"].double() if "mass" in s else None
    for i, length in enumerate(t):
        q = s["q"][i].double().view(c["n_kv"], G, D)
        z = torch.einsum("hgd,htd->hgt", q, _exact_rows(s, "k", i, length)) / math.sqrt(D)
        w = torch.softmax(z, dim=2)
        lse[i] = torch.logsumexp(z, dim=2).flatten()
        out[i] = torch.einsum("hgt,htd->hgd", w, _exact_rows(s, "v", i, length)).reshape(c["n_q"], D)
        if res is not None:
            pages, old = _exact_mass(s, i, length)
            old[:, -1] = 0
            _put_mass(res, s, pages, old + w.sum(dim=1))
    return {"out": out, "lse": lse} if res is None else {"out": out, "lse": lse, "mass": res}


def _exact_prompt(c, s):
    t, m, _, _ = _lens(c)
    G, at, res = c["n_q"] // c["n_kv"], 0, s["mass"].double()
    for i, (length, new) in enumerate(zip(t, m)):
        k = _exact_rows(s, "k", i, length)
        pages, w = _exact_mass(s, i, length)
        w[:, length - new if c["add"] else 0:] = 0
        for a in range(0, new, 512):
            b = min(new, a + 512)
            last = length - new + torch.arange(a, b, device=DEV)
            for h in range(c["n_kv"]):
                q, ls = (s[x][at + a:at + b, h * G:(h + 1) * G].double() for x in ("q", "lse"))
                z = torch.einsum("mgd,td->mgt", q, k[h]) / math.sqrt(D) - ls[..., None]
                z = z.masked_fill((torch.arange(length, device=DEV)[None, :] > last[:, None])[:, None], -math.inf)
                w[h] += torch.exp(z).sum(dim=(0, 1))
        _put_mass(res, s, pages, w)
        at += new
    return {"mass": res}


def _exact_evict(c, s):
    t, _, _, _ = _lens(c)
    P, H = c["page"], c["n_kv"]
    res = {x: s[x].double() if s[x] is not None else None for x in ("k_pages", "v_pages", "k_scale", "v_scale", "mass")}
    kept = s["kept"].clone()
    for i, (length, k) in enumerate(zip(t, _kept(c))):
        pages, w = _exact_mass(s, i, length)
        lo, hi = min(length, c["first"]), max(min(length, c["first"]), length - c["recent"])
        rows = {x: _exact_rows(s, x, i, length) for x in ("k", "v")}
        for h in range(H):
            if k == length:
                kept[i, h, :k] = torch.arange(k, device=DEV)
                continue
            # Heaviest first, the lower token first among equals.
            order = sorted(range(lo, hi), key=w[h].tolist().__getitem__, reverse=True)
            got = torch.tensor(sorted(list(range(lo)) + order[:k - lo - (length - hi)] + list(range(hi, length))), device=DEV)
            kept[i, h, :k] = got
            first = int((got == torch.arange(k, device=DEV)).long().cumprod(0).sum())        # tokens that stay in place
            for j in range(first // P, -(-k // P)):
                a, b = j * P, min(k, (j + 1) * P)
                if first >= b:
                    continue
                res["mass"][0, pages[j], h, :b - a] = w[h, got[a:b]]
                for x in ("k", "v"):
                    y = rows[x][h, got[a:b]]
                    if c["kv"] == "e4m3":
                        one = 2.0 ** max(-64, math.ceil(math.log2(float(y.abs().max()) / 448 or 2.0 ** -64)))
                        res[x + "_scale"][0, pages[j], h] = one
                        y = _e4m3(y / one)
                    res[x + "_pages"][0, pages[j], h, :b - a] = y
    return {"k": res["k_pages"], "v": res["v_pages"], "k_scale": res["k_scale"], "v_scale": res["v_scale"], "mass": res["mass"],
            "kept": kept, "new_len": s["kv_len"].clamp(max=s["keep"])}


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "evict":
        # Page by page: too long for the largest batches.
        return _exact_evict(c, s) if sum(_kept(c)) * c["n_kv"] // c["page"] <= 20000 else None
    return _exact_prompt(c, s) if c["op"] == "prompt" else _exact_attention(c, s)
