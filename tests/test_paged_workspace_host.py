"""Paged decode workspaces, without a GPU."""

import pytest

import attention_attn_fwd_bwd_gb300 as af
from tests.test_paged_host import FAKE, WS_SMALL, _cache, _decode


@pytest.fixture(scope="module")
def lib():
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    return af.load()


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 2), (64, 2)])
def test_each_cache_format_has_a_size_of_its_own(lib, Hq, Hkv):
    """A buffer of the smaller size is refused with a cache of the other format."""
    sizes = [af.paged_decode_workspace_size(Hq, Hkv, 128, f) for f in (af.CACHE_BF16, af.CACHE_Q4)]
    for q4, n in enumerate(sizes):
        assert _decode(lib, _cache(bool(q4)), Hq=Hq, ws_n=n - 1) == WS_SMALL
    if min(sizes) < max(sizes):
        assert _decode(lib, _cache(sizes[1] > sizes[0]), Hq=Hq, ws=FAKE, ws_n=min(sizes)) == WS_SMALL
