"""GPU: what a row does not see has no effect on its bits."""
import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af
from tests.test_gpu_paged import i32, make_cache, randn
from tests.test_gpu_paged_attend import run

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [2, 50])  # with groups of 4, a row tile and two
@pytest.mark.parametrize("theta", [None, 1e4])
def test_earlier_rows_keep_their_bits(q4, d, N, theta):
    """Calls that differ in the chunk's last key and value only, by 2^20. (A 4-bit tile is put under a power of
    two of its largest step. Keys keep all of their bits under it, down to steps of 2^-28, and scores change
    by that power of two and nothing else.)"""
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    cache = make_cache([300 + N], 2, 16, d, q4, seed=66, garbage=False)
    q = randn(1, 8, N, d, seed=67)
    k, v = randn(1, 2, 1, d, seed=68), randn(1, 2, 1, d, seed=69)
    got = []
    for size in (1.0, 2.0 ** 20):
        af.paged_append(cache, k * size, v * size, i32([300 + N - 1]), rope_mode=af.ROPE_NONE)
        got.append(run(q, cache, [300], None, theta))
    for a, b in zip(*got):
        assert torch.equal(a[:, :, :-1], b[:, :, :-1])
        assert not torch.equal(a[:, :, -1], b[:, :, -1])
