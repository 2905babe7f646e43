"""GPU: sizes of paged calls that are refused before a launch."""
import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
DEV = torch.device("cuda")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    af.load()
    assert af.device_status() == 0


def small(q4=False):
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=DEV)
    cache = af.PagedCache.empty(4, 2, 16, 64, table, q4=q4)
    for x in cache._tensors:
        if x is not None and x is not table:
            x.zero_()
    return cache


@pytest.mark.parametrize("window", [-1, -(1 << 31), -(1 << 32), -(1 << 32) + 5, -(1 << 40)])
def test_negative_windows_of_any_size(window):
    """Those past 32 bits do not wrap into a valid one."""
    cache = small()
    q, lens = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises(af.AttnfuseError) as e:
        af.paged_decode(q, cache, lens, window=window)
    assert e.value.code == 1


@pytest.mark.parametrize("N", [2.5, 3.0, "3", None])
def test_a_gathers_row_count_is_a_whole_number(N):
    """A fraction is not cut off."""
    with pytest.raises(TypeError):
        af.paged_gather(small(), None, None, N)
