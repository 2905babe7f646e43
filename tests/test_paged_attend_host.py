"""Attention of a chunk over a paged cache, without a GPU: what the C entry points refuse."""
import ctypes

import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
FAKE = 0x100000  # 16-byte aligned, never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    return af.load()


def _st(*v):
    return (ctypes.c_int64 * len(v))(*v)


QS = _st(8 * 5 * 128, 5 * 128, 128, 1)


def _cache(q4=False, **kw):
    c = af.CPagedCache()
    c.format, c.num_pages, c.Hkv, c.page_size, c.d, c.B, c.max_pages = int(q4), 10, 2, 16, 128, 3, 4
    row = 64 if q4 else 128
    c.k = c.v = FAKE
    c.k_strides = c.v_strides = _st(2 * 16 * row, 16 * row, row, 1)
    if q4:
        c.k_scales = c.v_scales = FAKE
        c.k_scale_strides = c.v_scale_strides = _st(2 * 16 * 4, 16 * 4, 4, 1)
    c.page_table, c.page_table_stride = FAKE, 4
    for n, v in kw.items():
        setattr(c, n, v)
    return c


def _attend(lib, c, q=FAKE, qs=QS, start=FAKE, count=None, out=FAKE, os=QS, lse=None, Hq=8, N=5, scale=0.1, theta=1e4, mode=1,
            window=0, slopes=None, ws=FAKE, ws_n=1 << 40):
    return lib.attnfuse_paged_attend(None if c is None else ctypes.byref(c), q, qs, start, count, out, os, lse, Hq, N, scale, theta,
                                     mode, window, slopes, ws, ws_n, None)


@pytest.mark.parametrize("kw, want", [
    (dict(format=2), INVALID), (dict(num_pages=0), INVALID), (dict(B=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(page_size=24), UNSUPPORTED), (dict(max_pages=(1 << 20) + 1), UNSUPPORTED), (dict(v=FAKE + 8), INVALID),
    (dict(page_table=0), INVALID)])
def test_cache_is_checked(lib, kw, want):
    assert _attend(lib, _cache(**kw)) == want
    assert lib.attnfuse_last_error() != b""


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("kw, want", [
    (dict(q=0), INVALID), (dict(q=FAKE + 8), INVALID), (dict(qs=_st(8 * 5 * 128, 5 * 128, 132, 1)), INVALID),
    (dict(qs=_st(8 * 5 * 128, 5 * 128, 128, 2)), INVALID), (dict(start=0), INVALID), (dict(start=FAKE + 2), INVALID),
    (dict(count=FAKE + 1), INVALID), (dict(out=0), INVALID), (dict(out=FAKE + 2), INVALID), (dict(os=_st(8 * 5 * 128, 0, 128, 1)), INVALID),
    (dict(lse=FAKE + 2), INVALID), (dict(Hq=7), UNSUPPORTED), (dict(Hq=0), INVALID), (dict(Hq=8192), UNSUPPORTED), (dict(N=0), INVALID),
    (dict(N=1 << 30), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(theta=-1.0), INVALID),
    (dict(theta=float("inf")), INVALID), (dict(mode=2), UNSUPPORTED), (dict(window=-1), INVALID), (dict(slopes=FAKE + 1), INVALID)])
def test_arguments_are_checked(lib, q4, kw, want):
    assert _attend(lib, _cache(q4), **kw) == want


def test_null_cache_is_refused(lib):
    assert _attend(lib, None) == INVALID


def test_workspace_size(lib):
    n = ctypes.c_size_t()
    size = lambda *a: lib.attnfuse_paged_attend_workspace_size(*a, ctypes.byref(n))  # noqa: E731
    assert size(3, 8, 2, 5, 128, 0, 1) == OK
    for bad, want in (((0, 8, 2, 5, 128, 0, 1), INVALID), ((3, 0, 2, 5, 128, 0, 1), INVALID), ((3, 8, 2, 0, 128, 0, 1), INVALID),
                      ((3, 8, 3, 5, 128, 0, 1), UNSUPPORTED), ((3, 8, 2, 5, 80, 0, 1), UNSUPPORTED), ((3, 8, 2, 5, 128, 2, 1), INVALID),
                      ((3, 8, 2, 5, 128, 0, 2), UNSUPPORTED), ((1 << 20, 4096, 1, 5, 128, 0, 1), UNSUPPORTED)):
        assert size(*bad) == want, bad
    assert lib.attnfuse_paged_attend_workspace_size(3, 8, 2, 5, 128, 0, 1, None) == INVALID


def test_binding_refuses_what_is_no_cache():
    with pytest.raises(TypeError):
        af.paged_attend(torch.zeros(1, 2, 3, 64).bfloat16(), None, None)
