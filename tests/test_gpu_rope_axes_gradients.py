"""GPU: gradients of the rope_axes stage, element by element: those of the backward at the rotated rows,
rounded to bf16, turned back and rounded again, and nothing else."""
import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af
from attention_attn_fwd_bwd_gb300 import combinators as C
from tests.test_gpu_rope_axes import angles, check, positions, randn

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("d, sections, interleaved, own", [(64, (32,), False, False), (64, (16, 16), True, True), (128, (16, 24, 24), False, False)])
@pytest.mark.parametrize("Hq, Hk", [(4, 4), (6, 2)])
def test_gradients_are_the_backwards_turned_back(d, sections, interleaved, own, Hq, Hk):
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    B, N = 2, 150
    q, k, v = (randn(B, h, N, d, seed=50 + i).requires_grad_() for i, h in enumerate((Hq, Hk, Hk)))
    dout = randn(B, Hq, N, d, seed=53)
    pos = positions(len(sections), B, N, -20, 400, 54)
    attn = C.attention(C.rope_axes(pos, sections, theta=1e4, interleaved=interleaved, own_spectrum=own), C.causal())
    out = attn(q, k, v)
    dq, dk, dv = torch.autograd.grad(out, (q, k, v), dout)
    with torch.no_grad():
        how = dict(rope_theta=1e4, interleaved=interleaved, own_spectrum=own)
        rq, rk = af.rope_axes(q, k, pos, sections, **how)
        var = af.Variant(mask=af.MASK_CAUSAL)
        o, lse = af.fwd(rq, rk, v, rope_mode=af.ROPE_NONE, variant=var)
        gq, gk, gv = af.bwd(rq, rk, v, o, lse, dout, rope_mode=af.ROPE_NONE, variant=var)
        assert torch.equal(out, o) and torch.equal(dv, gv)
        back = -angles(pos, sections, 1e4, interleaved, own)
        # beside the backward's own rounding (of gq, gk) one of half a step
        check(dq, gq, back, 400 * 2.0 ** -51), check(dk, gk, back, 400 * 2.0 ** -51)
        tq, tk = af.rope_axes(gq, gk, pos, sections, inverse=True, **how)
        assert torch.equal(dq, tq) and torch.equal(dk, tk)
    assert af.device_status() == 0
