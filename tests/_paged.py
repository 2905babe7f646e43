"""Plain 64-bit statements of the paged-cache operators, for the tests (torch, any device)."""
import math

import torch

GROUP = 32


def rotated(x, pos, theta):
    """R_p x in 64 bits: x [..., n, d], pos [n] or broadcastable to x[..., 0]."""
    x = x.double()
    d = x.shape[-1]
    i = torch.arange(d // 2, dtype=torch.float64, device=x.device)
    a = pos.to(x.device).double()[..., None] * float(theta) ** (-2.0 * i / d)
    c, s = torch.cos(a), torch.sin(a)
    lo, hi = x[..., : d // 2], x[..., d // 2:]
    return torch.cat((lo * c - hi * s, hi * c + lo * s), -1)


def as_row(x64):
    """What a bf16 cache holds of an exact value: rounded to fp32, then to bf16."""
    return x64.float().bfloat16()


def quantised(row):
    """bf16 [..., d] -> (codes int [..., d], steps bf16 [..., d/32])."""
    g = row.double().unflatten(-1, (-1, GROUP))
    a = g.abs().amax(-1)
    step = (a.float() / 7).bfloat16()
    bad = ~torch.isfinite(g).all(-1)
    step[a < 2.0 ** -96] = 0
    step[bad] = math.nan
    live = (step > 0) & ~bad
    t = g / torch.where(live, step.double(), torch.ones_like(a))[..., None]
    code = torch.where(t < 0, -torch.floor(-t + 0.5), torch.floor(t + 0.5)).clamp(-7, 7)
    code = torch.where(live[..., None], code, torch.zeros_like(code))
    return code.flatten(-2).to(torch.int64), step


def nibble_of(c, slot, d):
    """Nibble (from the row's first byte on) that holds element c of a slot's row."""
    g, r, i = c // 32, (c % 32) // 4, c % 4
    if d == 128 and slot & 2:
        r ^= 4
    return 4 * (r * (d // 32) + g) + i


def row_nibbles(page, d):
    return torch.tensor([[nibble_of(c, s, d) for c in range(d)] for s in range(page)])


def packed(codes):
    """Codes [P, H, page, d] -> uint8 [P, H, page, d/2] as the cache stores them."""
    P, H, S, d = codes.shape
    at = row_nibbles(S, d).to(codes.device).expand(P, H, S, d)
    nib = torch.zeros_like(codes).scatter_(3, at, codes + 8)
    return (nib[..., 0::2] | (nib[..., 1::2] << 4)).to(torch.uint8)


def unpacked(rows):
    P, H, S, w = rows.shape
    d = 2 * w
    nib = torch.stack((rows & 15, rows >> 4), -1).flatten(3).long()
    return torch.gather(nib, 3, row_nibbles(S, d).to(rows.device).expand(P, H, S, d)) - 8


def values(cache, which):
    """The whole pool's values in 64 bits, [P, Hkv, page, d]."""
    pool = getattr(cache, which)
    if not cache.q4:
        return pool.double()
    steps = getattr(cache, which + "_scales").double()
    return unpacked(pool).double() * steps.repeat_interleave(GROUP, -1)


def rows(pool64, table, b, first, n):
    """Positions first .. first + n - 1 of sequence b: [Hkv, n, d]."""
    S = pool64.shape[2]
    p = torch.arange(first, first + n, device=pool64.device)
    return pool64[table[b, p // S].long(), :, p % S].transpose(0, 1)


def decode(q, cache, lens, scale, theta=None, window=0, slopes=None):
    """(out, lse, tol_out, tol_lse) in 64 bits: [B, Hq, d] and [B, Hq].

    tol_lse: a score may be off by ds = 2^-15 scale sum|q_i||k_i| (q in two bf16 parts keeps 2^-17
    of each product, fp32 sums of 128 products and the centring of 4-bit codes take less than
    that again) plus 2^-22 of the score's and the bias' size, and the sum by 2^-20.
    tol_out: half a step of bf16, 2^-8 |o|, plus the weights' rounding to fp16 or finer, 2^-11, and
    twice the score's error, each on sum p|v|."""
    B, Hq, d = q.shape
    k64, v64 = values(cache, "k"), values(cache, "v")
    Hkv = cache.Hkv
    out = torch.zeros(B, Hq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    tol_out, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b, L in enumerate(lens.tolist()):
        if L == 0:
            continue
        first = max(0, L - window) if window else 0
        qb = q[b].double()
        if theta is not None:
            qb = rotated(qb, torch.tensor(L - 1), theta)
        qb = qb.view(Hkv, -1, d)
        k, v = (rows(x, cache.page_table, b, first, L - first) for x in (k64, v64))
        x = scale * torch.einsum("hgc,hnc->hgn", qb, k)
        size = scale * torch.einsum("hgc,hnc->hgn", qb.abs(), k.abs())
        bias = torch.zeros_like(x)
        if slopes is not None:
            n = torch.arange(first, L, device=q.device)
            bias = slopes.double().view(Hkv, -1, 1) * (n - (L - 1))
        x = x + bias
        l = torch.logsumexp(x, -1)
        p = torch.exp(x - l[..., None])
        ds = 2.0 ** -15 * size + 2.0 ** -22 * (x.abs() + bias.abs())
        ds = torch.where(p > 2.0 ** -40, ds, torch.zeros_like(ds)).amax(-1)
        out[b] = torch.einsum("hgn,hnc->hgc", p, v).reshape(Hq, d)
        lse[b] = l.view(-1)
        tol_lse[b] = (ds + 2.0 ** -20 * (1 + l.abs())).view(-1)
        pv = torch.einsum("hgn,hnc->hgc", p, v.abs())
        tol_out[b] = (2.0 ** -8 * out[b].view(Hkv, -1, d).abs() + (2.0 ** -11 + 2 * ds[..., None]) * pv).view(Hq, d)
    return out, lse, tol_out, tol_lse


def check_decode(got, ref):
    (out, lse), (o, l, to, tl) = got, ref
    assert torch.isfinite(out).all(), "non-finite output"
    err = (out.double() - o).abs() - to
    assert err.max().item() <= 0, f"out: {err.max().item():.3e} over its tolerance"
    none = torch.isinf(l)
    assert torch.equal(torch.isinf(lse), none) and (lse[none] < 0).all() and not torch.isnan(lse).any()
    err = torch.where(none, torch.zeros_like(l), (lse.double() - l).abs() - tl)
    assert err.max().item() <= 0, f"lse: {err.max().item():.3e} over its tolerance"
