"""Decodes, dense and paged, from a cold cache: tiles then arrive late and in any order, and every
repetition still gives the same bits."""
import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af
from attention_attn_fwd_bwd_gb300 import inputs

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    af.load()
    assert af.device_status() == 0


def _repeat(call, times=60):
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")  # more than the L2 holds
    first = [x.clone() for x in call()]
    for i in range(times):
        flush.fill_(i & 255)
        for x, y in zip(call(), first):
            assert torch.equal(x, y), f"repetition {i}: {(x != y).sum().item()} of {x.numel()} values differ"
    assert af.device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L,B", [(4096, 8), (16384, 1)])
def test_dense_decode_from_a_cold_cache(L, B, d):
    x = inputs.decode(B, 32, 8, L, d, seed=90 + L + B)
    q, k, v = (x[n].cuda() for n in ("q", "k_cache", "v_cache"))
    _repeat(lambda: af.decode(q, k, v, L - 1, rope_theta=5e5))


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("L,B", [(4096, 8), (16384, 1)])
def test_paged_decode_from_a_cold_cache(L, B, q4):
    x = inputs.decode(B, 32, 8, L, 128, seed=91 + L + B)
    q, k, v = (x[n].cuda() for n in ("q", "k_cache", "v_cache"))
    pages = -(-L // 64)
    table = torch.randperm(B * pages, generator=torch.Generator().manual_seed(92)).int().view(B, pages).cuda()
    cache = af.PagedCache.empty(B * pages, 8, 64, 128, table, q4=q4)
    zero, lens = (torch.full((B,), n, dtype=torch.int32, device="cuda") for n in (0, L))
    af.paged_append(cache, k, v, zero, rope_mode=af.ROPE_NONE)
    _repeat(lambda: af.paged_decode(q, cache, lens, rope_theta=5e5))
