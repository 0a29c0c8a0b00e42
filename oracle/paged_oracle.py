"""The paged cache's operators in 64 bits, from their definitions (test infrastructure, never on the product path).

Works on torch tensors of any device; every sum, exponential and rotation is in float64, and the e4m3 rounding is
done on doubles (nearest value, ties to the even code), not by a conversion of a library.
"""
from __future__ import annotations

import math

import torch

D = 128


def e4m3_values():
    """The 127 finite non-negative values in code order: subnormals k 2^-9, then (8 + m) 2^(e - 10), up to 448."""
    vals = [k * 2.0 ** -9 for k in range(8)]
    vals += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return vals[:127]            # code 127 is NaN


def e4m3_round(x):
    """Nearest e4m3 value of doubles, ties to the even code, saturating at 448; NaN stays NaN."""
    a = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -30))).clamp(min=-6.0) - 3.0)
    return torch.round(a / step) * step * torch.sign(x)


def scale_of(amax):
    """Smallest power of two, at least 2^-64, with amax <= 448 times it (a double)."""
    s = 2.0 ** -64
    while amax > 448.0 * s:
        s *= 2.0
    return s


def rotate(x, pos, table, rot, interleaved):
    """x: double [n, heads, 128]; the first rot channels turned by the table's angles of each row's position."""
    y = x.clone()
    h = rot // 2
    if not h:
        return y
    c, s = table[pos].double()[:, None, :h], table[pos].double()[:, None, h:]
    i = torch.arange(h, device=x.device)
    p, r = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    y[..., p] = x[..., p] * c - x[..., r] * s
    y[..., r] = x[..., r] * c + x[..., p] * s
    return y


def append_page(codes, scale, y, s0):
    """One page of one head after y (double [m, 128]) went into its slots s0.. : (codes as doubles [P, 128], scale)."""
    fine = y.abs()[torch.isfinite(y)]
    s = scale_of(float(fine.max()) if fine.numel() else 0.0)
    codes = codes.clone()
    if s0 > 0 and scale >= s:
        s = scale
    elif s0 > 0:
        codes[:s0] = e4m3_round(codes[:s0] * (scale / s))
    codes[s0:s0 + y.shape[0]] = e4m3_round(y / s)
    return codes, s


def attention(q, k, v, scale, n_see):
    """q: [m, d], k, v: [T, d] doubles; row j sees the first n_see[j] keys.  (out, lse, weighted |v|, largest
    scale sum |q k|): the last two are what error bounds are made of."""
    m, T = q.shape[0], k.shape[0]
    if T == 0:
        z = torch.zeros(m, D, dtype=torch.float64, device=q.device)
        return z, torch.full((m,), -math.inf, dtype=torch.float64, device=q.device), z, z[:, 0]
    z = q @ k.T * scale
    hid = torch.arange(T, device=q.device)[None, :] >= n_see[:, None]
    z = z.masked_fill(hid, -math.inf)
    top = z.amax(dim=1, keepdim=True)
    none = torch.isinf(top) & (top < 0)
    w = torch.where(hid, torch.zeros_like(z), torch.exp(z - torch.where(none, torch.zeros_like(top), top)))
    tot = w.sum(dim=1, keepdim=True)
    p = w / torch.where(none, torch.ones_like(tot), tot)
    lse = torch.where(none, top, top + torch.log(tot))[:, 0]
    big = (q.abs() @ k.abs().T * abs(scale)).masked_fill(hid, 0).amax(dim=1)
    return p @ v, lse, p @ v.abs(), big


def mass(q, k, scale, n_see, lse=None):
    """q: [m, d], k: [T, d] doubles; row j sees the first n_see[j] keys.  (sum over rows of exp(logit - lse) per key,
    the same with each weight times its row's largest scale sum |q k| plus |lse|: what error bounds are made of.)
    lse [m]: the rows' (default: their own)."""
    T = k.shape[0]
    if T == 0 or q.shape[0] == 0:
        z = torch.zeros(T, dtype=torch.float64, device=k.device)
        return z, z
    hid = torch.arange(T, device=q.device)[None, :] >= n_see[:, None]
    z = (q @ k.T * scale).masked_fill(hid, -math.inf)
    if lse is None:
        lse = torch.logsumexp(z, dim=1)
    none = torch.isinf(lse) & (lse < 0)
    w = torch.where(hid | none[:, None], torch.zeros_like(z), torch.exp(z - torch.where(none, torch.zeros_like(lse), lse)[:, None]))
    big = (q.abs() @ k.abs().T * abs(scale)).masked_fill(hid, 0).amax(dim=1) + torch.where(none, torch.zeros_like(lse), lse).abs()
    return w.sum(dim=0), (w * big[:, None]).sum(dim=0)


def evict_tokens(w, keep, first, recent):
    """Numbers, ascending, of the tokens of one head that stay; w: the masses of all held tokens (NaN: below all)."""
    T = len(w)
    if T <= keep:
        return list(range(T))
    mid = range(first, T - recent)
    best = sorted(mid, key=lambda t: (w[t] != w[t], 0.0 if w[t] != w[t] else -w[t], t))[:keep - first - recent]
    return list(range(first)) + sorted(best) + list(range(T - recent, T))
