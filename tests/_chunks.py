"""Plain 64-bit statement of the attention of a chunk over a paged cache, for the tests."""
import math

import torch

from tests import _paged as P


def attend(q, cache, start, count, scale, theta=None, window=0, slopes=None):
    """(out, lse, tol_out, tol_lse) in 64 bits: [B, Hq, N, d] and [B, Hq, N]; start, count: lists.

    tol_lse: a score may be off by ds = 2^-15 scale sum|q_i||k_i| (q in two bf16 parts keeps 2^-16
    of each product, fp32 sums of 128 products take less than that again) plus 2^-22 of the score's
    and the bias' size, and the sum by 2^-20.
    tol_out: half a step of bf16, 2^-8 |o|, plus the weights' rounding to bf16, 2^-8, the same for the
    values of a 4-bit cache, and twice the score's error, each on sum p|v|; and 2^-125 sum|v|, since
    weights are 32-bit floats: one below 2^-126 of the largest (an exponential's smallest normal
    result), or of a part's largest with the part's own below 2^-126 of the whole's, may be 0, which takes
    at most 2 * 2^-126 |v| from the sum. (Found by values that underflow: weights e^-370 and no other
    key with a code other than 0 in that element.)"""
    B, Hq, N, d = q.shape
    k64, v64 = P.values(cache, "k"), P.values(cache, "v")
    Hkv = cache.Hkv
    f64 = dict(dtype=torch.float64, device=q.device)
    out, lse = torch.zeros(B, Hq, N, d, **f64), torch.full((B, Hq, N), -math.inf, **f64)
    tol_out, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    round_v = 2.0 ** -8 if cache.q4 else 0.0
    for b in range(B):
        n = count[b]
        if not n:
            continue
        p0, end = start[b], start[b] + n
        first = max(0, p0 - window + 1) if window else 0
        pos = torch.arange(p0, end, device=q.device)
        m = torch.arange(first, end, device=q.device)
        qb = q[b, :, :n].double()
        if theta is not None:
            qb = P.rotated(qb, pos, theta)
        qb = qb.reshape(Hkv, -1, n, d)
        k, v = (P.rows(x, cache.page_table, b, first, end - first) for x in (k64, v64))
        x = scale * torch.einsum("hgic,hnc->hgin", qb, k)
        size = scale * torch.einsum("hgic,hnc->hgin", qb.abs(), k.abs())
        bias = torch.zeros_like(x)
        if slopes is not None:
            bias = slopes.double().view(Hkv, -1, 1, 1) * (m - pos[:, None])
        seen = m <= pos[:, None]
        if window:
            seen &= m > pos[:, None] - window
        x = (x + bias).masked_fill(~seen, -math.inf)
        l = torch.logsumexp(x, -1)
        w = torch.exp(x - l[..., None])
        ds = 2.0 ** -15 * size + 2.0 ** -22 * (x.abs() + bias.abs())
        ds = torch.where(w > 2.0 ** -40, ds, torch.zeros_like(ds)).amax(-1)
        o = torch.einsum("hgin,hnc->hgic", w, v)
        out[b, :, :n] = o.reshape(Hq, n, d)
        lse[b, :, :n] = l.view(Hq, n)
        tol_lse[b, :, :n] = (ds + 2.0 ** -20 * (1 + l.abs())).view(Hq, n)
        pv = torch.einsum("hgin,hnc->hgic", w, v.abs())
        none = 2.0 ** -125 * v.abs().sum(1)[:, None, None]
        tol_out[b, :, :n] = (2.0 ** -8 * o.abs() + (2.0 ** -8 + round_v + 2 * ds[..., None]) * pv + none).view(Hq, n, d)
    return out, lse, tol_out, tol_lse


def check(got, ref):
    (out, lse), (o, l, to, tl) = got, ref
    assert torch.isfinite(out).all(), "non-finite output"
    err = (out.double() - o).abs() - to
    assert err.max().item() <= 0, f"out: {err.max().item():.3e} over its tolerance"
    if lse is None:
        return
    none = torch.isinf(l)
    assert torch.equal(torch.isinf(lse), none) and (lse[none] < 0).all() and not torch.isnan(lse).any()
    err = torch.where(none, torch.zeros_like(l), (lse.double() - l).abs() - tl)
    assert err.max().item() <= 0, f"lse: {err.max().item():.3e} over its tolerance"
