"""Rotary positions on several axes, without a GPU: what the C entry point and the binding refuse."""
import ctypes

import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af
from attention_attn_fwd_bwd_gb300 import combinators as C

INVALID, UNSUPPORTED = 1, 2
FAKE = 0x100000  # 16-byte aligned, never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    return af.load()


def _st(*v):
    return (ctypes.c_int64 * len(v))(*v)


QS, KS = _st(4 * 10 * 128, 10 * 128, 128, 1), _st(2 * 10 * 128, 10 * 128, 128, 1)


def _map(sections=(16, 24, 24), **kw):
    m = af.CRopeAxesMap()
    m.axes, m.rope_theta, m.positions = len(sections), 1e4, FAKE
    for i, n in enumerate(sections[:4]):
        m.sections[i] = n
    m.position_strides = _st(30, 10, 1)
    for n, v in kw.items():
        setattr(m, n, v)
    return m


def _call(lib, m, q=FAKE, qs=QS, qo=FAKE, k=FAKE, ks=KS, ko=FAKE, Hq=4, Hk=2, B=3, N=10, d=128):
    return lib.attnfuse_rope_axes(q, qs, qo, QS, Hq, k, ks, ko, KS, Hk, B, N, d, None if m is None else ctypes.byref(m), 0, None)


@pytest.mark.parametrize("kw, want", [
    (dict(sections=(16, 24, 23)), INVALID), (dict(sections=(16, 0, 48)), INVALID), (dict(sections=()), INVALID),
    (dict(sections=(16, 16, 16, 8, 8)), INVALID), (dict(sections=(64,), axes=-1), INVALID), (dict(sections=(80, -16)), INVALID),
    (dict(rope_theta=0.0), INVALID), (dict(rope_theta=float("nan")), INVALID), (dict(rope_theta=float("inf")), INVALID),
    (dict(positions=0), INVALID), (dict(positions=FAKE + 2), INVALID), (dict(position_strides=_st(30, -10, 1)), INVALID)])
def test_map_is_checked(lib, kw, want):
    assert _call(lib, _map(**kw)) == want
    assert lib.attnfuse_last_error() != b""


@pytest.mark.parametrize("kw, want", [
    (dict(q=0), INVALID), (dict(q=FAKE + 8), INVALID), (dict(qo=0), INVALID), (dict(k=0), INVALID), (dict(ko=FAKE + 2), INVALID),
    (dict(qs=_st(4 * 10 * 128, 10 * 128, 132, 1)), INVALID), (dict(ks=_st(2 * 10 * 128, 10 * 128, 128, 2)), INVALID),
    (dict(qs=_st(0, 10 * 128, 128, 1)), INVALID), (dict(d=96), UNSUPPORTED), (dict(Hq=0), INVALID), (dict(Hk=-1), INVALID),
    (dict(Hq=4097), UNSUPPORTED), (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(B=1 << 16, N=1 << 16), UNSUPPORTED)])
def test_tensors_are_checked(lib, kw, want):
    assert _call(lib, _map(), **kw) == want


def test_null_map_is_refused(lib):
    assert _call(lib, None) == INVALID


def test_binding_refuses_cpu_tensors_and_other_types():
    q = torch.zeros(1, 4, 10, 128)
    pos = torch.zeros(3, 1, 10, dtype=torch.int32)
    with pytest.raises(TypeError):
        af.rope_axes(q, None, pos, (16, 24, 24))
    with pytest.raises(ValueError):
        af.rope_axes(q.bfloat16(), None, pos, (16, 24, 24))
    with pytest.raises(TypeError):
        af.rope_axes(None, None, pos, (16, 24, 24))


def test_combinator_stands_alone_with_its_rotation():
    pos = torch.zeros(2, 10, dtype=torch.int32)
    a = C.attention(C.rope_axes(pos, (32, 32)), C.causal())
    assert a.rope_mode == af.ROPE_NONE and a.axes["sections"] == (32, 32)
    with pytest.raises(ValueError):
        C.attention(C.rope(), C.rope_axes(pos, (32, 32)))
