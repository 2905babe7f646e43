"""Chunks over a 4-bit cache whose outputs show the rounding of the weights and little else, for the tests.

Values are codes times powers of two, exact in bf16. Neighbouring positions 2i and 2i + 1 have nearly the
same key and opposite values, so that an output is much smaller than sum p|v|: its own rounding to
bf16 is small beside that of the weights, which does not cancel."""
import math

import torch

from tests import _paged as P

Hkv, G, PAGE = 2, 4, 16


class Problem:
    def __init__(self, d, N, theta, window, start, seed, device):
        g = torch.Generator().manual_seed(seed)
        pages = [-(-(s + N) // PAGE) for s in start]
        n, wide = sum(pages), max(pages)
        shape = (n, Hkv, PAGE, d)
        self.d, self.N, self.theta, self.window, self.start = d, N, theta, window, start
        kc, vc = (torch.randint(-6, 7, shape, generator=g) for _ in "kv")
        kc[:, :, 1::2] = kc[:, :, 0::2]
        kc[:, :, 1::2, ::32] += 1
        vc[:, :, 1::2] = -vc[:, :, 0::2]
        self.ks = (0.1 + 0.05 * torch.rand(n, Hkv, PAGE // 2, d // 32, generator=g)).bfloat16().repeat_interleave(2, 2)
        self.vs = (2.0 ** torch.randint(-3, 4, (n, Hkv, 1, d // 32), generator=g)).bfloat16().expand(-1, -1, PAGE, -1).contiguous()
        order = torch.randperm(n, generator=g).to(torch.int32).tolist()
        self.table = torch.tensor([[order.pop() for _ in range(m)] + [-1] * (wide - m) for m in pages], dtype=torch.int32)
        self.q = (0.5 * torch.randn(len(start), Hkv * G, N, d, generator=g)).bfloat16()
        self.k64 = kc.double() * self.ks.double().repeat_interleave(32, -1)
        self.v64 = vc.double() * self.vs.double().repeat_interleave(32, -1)
        self.k, self.v = P.packed(kc), P.packed(vc)
        for name in ("ks", "vs", "table", "q", "k64", "v64", "k", "v"):
            setattr(self, name, getattr(self, name).to(device))

    def attend(self, weights):
        """(out, tolerance) in 64 bits, [B, Hq, N, d], of exp(x - max) -> weights(..) in the sum with the values.

        tolerance: half a step of bf16, 2^-8 |o|; on sum p|v|: two bf16 parts of a weight leave
        2^-8 2^-8 of it; 16 products (two parts of 128 keys, 16 at a time) add 17 numbers each, each
        cut at 2^-23 of the largest at most, 2^-14.9; another 2^-20 for sums and exponentials; and twice
        what a score is off by: 8 products of 16 elements, 16 where q is in two parts, the same way, 2^-15.9
        or 2^-14.9 of scale sum|q_i||k_i|, 2^-20 of it for the 22 bits of a rotated q, 2^-22 of the score."""
        B, d, N = len(self.start), self.d, self.N
        out = torch.zeros(B, Hkv * G, N, d, dtype=torch.float64, device=self.q.device)
        tol = torch.zeros_like(out)
        products = 16 if self.theta else 8
        for b, p0 in enumerate(self.start):
            end = p0 + N
            pos, m = (torch.arange(a, end, device=out.device) for a in (p0, 0))
            q = self.q[b].double()
            if self.theta:
                q = P.rotated(q, pos, self.theta)
            q = q.reshape(Hkv, G, N, d)
            k, v = (P.rows(x, self.table, b, 0, end) for x in (self.k64, self.v64))
            scale = d ** -0.5
            x = scale * torch.einsum("hgic,hnc->hgin", q, k)
            size = scale * torch.einsum("hgic,hnc->hgin", q.abs(), k.abs())
            seen = m <= pos[:, None]
            if self.window:
                seen &= m > pos[:, None] - self.window
            w = torch.exp(x.masked_fill(~seen, -math.inf) - x.masked_fill(~seen, -math.inf).amax(-1, keepdim=True))
            total = w.sum(-1, keepdim=True)
            o = torch.einsum("hgin,hnc->hgic", weights(w), v) / total
            pv = torch.einsum("hgin,hnc->hgic", w, v.abs()) / total
            ds = ((products * 17 * 2.0 ** -23 + 2.0 ** -20) * size + 2.0 ** -22 * x.abs()).masked_fill(~seen, 0).amax(-1, keepdim=True)
            out[b] = o.reshape(-1, N, d)
            tol[b] = (2.0 ** -8 * o.abs() + (2.0 ** -16 + 16 * 17 * 2.0 ** -23 + 2.0 ** -20 + 2 * ds) * pv).reshape(-1, N, d)
        return out, tol


CASES = [  # d, N (a row tile of 24 rows, two of 240), theta, window, starts
    (128, 6, None, 4, [31, 120, 1]), (128, 60, None, 4, [33, 100]), (64, 6, None, 4, [31, 120, 1]), (64, 60, None, 4, [33, 100]),
    (128, 6, 1e4, 4, [31, 120, 1]), (128, 60, 1e4, 4, [33, 100]), (64, 6, 1e4, 4, [31, 120, 1]), (64, 60, 1e4, 4, [33, 100]),
    (128, 6, None, 0, [5, 13, 21]), (128, 60, None, 0, [1, 9]), (64, 60, 1e4, 0, [1, 9]),
]
