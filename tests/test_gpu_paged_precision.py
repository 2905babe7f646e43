"""GPU: how many bits of a rotated query the paged decode keeps, read off single scores."""
import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af
from tests import _paged as P

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
DEV = torch.device("cuda")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    af.load()
    assert af.device_status() == 0


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d", [(32, 8, 128), (8, 1, 128), (32, 2, 128), (32, 4, 64), (2, 1, 64)])
def test_a_score_keeps_the_querys_bits(q4, Hq, Hkv, d):
    """One pair (x, y) of a query is not zero, nor is one element of the last key, which belongs to
    that pair; the earlier keys score -200 or less by a slope. So the log-sum-exp is one product,
    scale x' k, and shows x' = x c - y s: off by at most 2^-20 (|x| + |y|) scale |k|.

    That bar, in roundings of 2^-24 relative to (|x| + |y|) or to what follows from it: c and s to
    fp32 1, the rotation's product and sum 2, the parts of q 2 (three of bf16: 2^-25; two of fp16:
    2^-23), the products' sum 2 (a 4-bit code enters as code + 8 with 8 taken out, so up to twice
    the score stands in between: 4 in all), scale * log2(e) 2, the product with it 1, ln 2 and its
    product 2: at most 14 < 16. Two parts of bf16 would leave 2^-18."""
    B, L, page, scale, theta = 64, 3, 16, 0.25, 1e4
    g = torch.Generator(DEV).manual_seed(d + Hq)
    pair = torch.randint(0, d // 2, (B, Hkv), generator=g, device=DEV)
    q = torch.zeros(B, Hkv, Hq // Hkv, d, device=DEV)
    xy = torch.randn(2, B, Hkv, Hq // Hkv, generator=g, device=DEV)
    at = pair[:, :, None, None].expand(-1, -1, Hq // Hkv, 1)
    q.scatter_(3, at, xy[0][..., None]).scatter_(3, at + d // 2, xy[1][..., None])
    q = q.view(B, Hq, d).bfloat16()
    which = torch.randint(0, 2, (B, Hkv), generator=g, device=DEV) * (d // 2)
    k = torch.zeros(B, Hkv, L, d, device=DEV)
    k[:, :, -1].scatter_(2, (pair + which)[..., None], 0.5 + torch.rand(B, Hkv, 1, generator=g, device=DEV))
    k = k.bfloat16()
    pages = torch.arange(B, dtype=torch.int32, device=DEV).view(B, 1)
    cache = af.PagedCache.empty(B, Hkv, page, d, pages, q4=q4)
    lens = torch.randint(L, page + 1, (B,), generator=g, device=DEV).int()  # the query's position
    af.paged_append(cache, torch.zeros(B, Hkv, page, d, device=DEV).bfloat16(),
                    torch.zeros(B, Hkv, page, d, device=DEV).bfloat16(), torch.zeros_like(lens))
    af.paged_append(cache, k, k, lens - L, rope_mode=af.ROPE_NONE)
    slopes = torch.full((Hq,), 200.0, device=DEV)
    out, lse = af.paged_decode(q, cache, lens, scale=scale, rope_theta=theta, alibi_slopes=slopes)
    torch.cuda.synchronize()
    assert af.device_status() == 0
    k64 = P.values(cache, "k")[pages[:, 0].long(), :, (lens - 1).long()]  # [B, Hkv, d]
    q64 = torch.stack([P.rotated(q[b], lens[b] - 1, theta) for b in range(B)]).view(B, Hkv, -1, d)
    want = scale * (q64 * k64[:, :, None]).sum(-1)
    size = scale * q.double().view_as(q64).abs().sum(-1) * k64.abs().amax(-1)[..., None]
    off = (lse.double().view_as(want) - want).abs() / size
    assert off.max().item() <= 2.0 ** -20, f"2^{off.max().log2().item():.2f}"
