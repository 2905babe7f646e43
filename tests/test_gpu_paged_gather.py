"""GPU: gathers large enough that a thread takes two heads, with the last head left over (odd Hkv),
against the cache's rows."""
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


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator(DEV).manual_seed(seed), device=DEV).bfloat16()


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv", [2, 3, 11])
def test_gather_of_two_heads_per_thread(q4, d, Hkv):
    """Rows * threads per row * heads past twice the GPU's slots; ragged counts, starts inside a
    page, one output a view between other data."""
    B, N, page, lens = 3, 9001, 48, [9001, 300, 9050]
    pages = -(-max(lens) // page)
    table = torch.randperm(B * pages, generator=torch.Generator().manual_seed(Hkv)).int().view(B, pages).to(DEV)
    cache = af.PagedCache.empty(B * pages, Hkv, page, d, table, q4=q4)
    for first in range(0, max(lens), 5000):  # every row of the cache, without the rotation
        n = min(5000, pages * page - first)
        af.paged_append(cache, randn(B, Hkv, n, d, seed=first), randn(B, Hkv, n, d, seed=first + 1), i32([first] * B),
                        rope_mode=af.ROPE_NONE)
    start, count = [0, 250, 49], [9001, 50, 9001]
    big = torch.full((B, Hkv, N, 2, d), 7.0, dtype=torch.bfloat16, device=DEV)
    k, v = af.paged_gather(cache, i32(start), i32(count), N, k=big[..., 0, :])
    torch.cuda.synchronize()
    assert af.device_status() == 0
    for got, which in ((k, "k"), (v, "v")):
        pool = P.values(cache, which)
        for b in range(B):
            want = P.rows(pool, table, b, start[b], count[b]).float().bfloat16()
            assert torch.equal(got[b, :, :count[b]], want)
            assert (got[b, :, count[b]:] == 0).all()
    assert (big[..., 1, :] == 7).all()
