"""GPU: a thread whose first CUDA call is one of the library's."""
import threading

import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def test_forward_and_backward_from_new_threads():
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    q, k, v = (torch.randn(1, 2, 200, 64, device="cuda").bfloat16() for _ in range(3))
    var = af.Variant(mask=af.MASK_CAUSAL)
    out, lse = af.fwd(q, k, v, rope_mode=af.ROPE_NONE, variant=var)
    want = af.bwd(q, k, v, out, lse, out, rope_mode=af.ROPE_NONE, variant=var)
    torch.cuda.synchronize()
    got, errors = {}, []

    def call(name, fn):
        try:
            got[name] = fn()
        except Exception as e:  # noqa: BLE001 - shown below
            errors.append(e)

    o, l, grads = torch.empty_like(out), torch.empty_like(lse), [torch.empty_like(q) for _ in range(3)]
    for name, fn in (("fwd", lambda: af.fwd(q, k, v, rope_mode=af.ROPE_NONE, variant=var, out=o, lse=l)),
                     ("bwd", lambda: af.bwd(q, k, v, out, lse, out, rope_mode=af.ROPE_NONE, variant=var,
                                            dq=grads[0], dk=grads[1], dv=grads[2]))):
        t = threading.Thread(target=call, args=(name, fn))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert torch.equal(got["fwd"][0], out) and torch.equal(got["fwd"][1], lse)
    assert all(torch.equal(a, b) for a, b in zip(got["bwd"], want))
