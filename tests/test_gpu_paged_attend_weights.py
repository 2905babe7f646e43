"""GPU parity: weights beside a 4-bit cache keep 16 bits (test_weights_host.py: with 8 these cases fail)."""
import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af
from tests import _weights as W

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("case", W.CASES)
def test_weights_keep_16_bits(case):
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    p = W.Problem(*case, seed=1, device=torch.device("cuda"))
    cache = af.PagedCache(p.k, p.v, p.table, p.ks, p.vs)
    start = torch.tensor(p.start, dtype=torch.int32, device="cuda")
    out, _ = af.paged_attend(p.q, cache, start, rope_theta=p.theta or 1e4,
                             rope_mode=af.ROPE_FUSED if p.theta else af.ROPE_NONE, window=p.window)
    torch.cuda.synchronize()
    assert af.device_status() == 0
    want, tol = p.attend(lambda w: w)
    err = (out.double() - want).abs() - tol
    assert err.max().item() <= 0, f"{err.max().item():.3e} over its tolerance"
