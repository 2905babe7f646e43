"""Paged caches, without a GPU: the C entry points refuse bad arguments before any CUDA call, the
binding refuses CPU tensors and other types, and the documented row format is a permutation."""
import ctypes

import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af
from tests import _paged as P

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
FAKE = 0x100000  # 16-byte aligned, never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    return af.load()


def _st(*v):
    return (ctypes.c_int64 * len(v))(*v)


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


X = _st(2 * 5 * 128, 5 * 128, 128, 1)


def _append(lib, c, k=FAKE, ks=X, start=FAKE, count=None, N=5, theta=1e4, mode=1):
    return lib.attnfuse_paged_append(ctypes.byref(c), k, ks, FAKE, X, start, count, N, theta, mode, None)


def _decode(lib, c, q=FAKE, qs=None, lens=FAKE, out=FAKE, Hq=8, scale=0.1, theta=1e4, mode=1, window=0, slopes=None,
            ws=FAKE, ws_n=1 << 30):
    return lib.attnfuse_paged_decode(ctypes.byref(c), q, qs or _st(8 * 128, 128, 1), lens, out, _st(8 * 128, 128, 1), None, Hq,
                                     scale, theta, mode, window, slopes, ws, ws_n, None)


@pytest.mark.parametrize("q4", [False, True])
def test_cache_descriptor_is_checked(lib, q4):
    row = 64 if q4 else 128
    for kw, want in ((dict(format=2), INVALID), (dict(num_pages=0), INVALID), (dict(Hkv=-1), INVALID), (dict(B=0), INVALID),
                     (dict(max_pages=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
                     (dict(page_size=24), UNSUPPORTED), (dict(page_size=1 << 17), UNSUPPORTED),
                     (dict(max_pages=(1 << 20) + 1), UNSUPPORTED), (dict(k=0), INVALID), (dict(v=FAKE + 8), INVALID),
                     (dict(page_table=0), INVALID), (dict(page_table=FAKE + 2), INVALID), (dict(page_table_stride=-4), INVALID),
                     (dict(k_strides=_st(2 * 16 * row, 16 * row, row, 2)), INVALID),
                     (dict(v_strides=_st(0, 16 * row, row, 1)), INVALID),
                     (dict(v_strides=_st(2 * 16 * row, 16 * row + 4, row, 1)), INVALID)):
        c = _cache(q4, **kw)
        assert _append(lib, c) == want, kw
        assert lib.attnfuse_last_error() != b""
        assert _decode(lib, c) == want, kw
        assert lib.attnfuse_paged_gather(ctypes.byref(c), None, None, FAKE, X, FAKE, X, 5, None) == want, kw
    assert lib.attnfuse_paged_append(None, FAKE, X, FAKE, X, FAKE, None, 5, 1e4, 1, None) == INVALID
    if q4:
        for kw in (dict(k_scales=0), dict(v_scales=FAKE + 4), dict(k_scale_strides=_st(2 * 16 * 4, 16 * 4, 8, 1)),
                   dict(v_scale_strides=_st(2 * 16 * 4 + 4, 16 * 4, 4, 1)), dict(k_strides=_st(2 * 16 * 64, 64, 2 * 64, 1))):
            assert _append(lib, _cache(True, **kw)) == INVALID, kw


def test_append_and_gather_arguments_are_checked(lib):
    c = _cache()
    for kw, want in ((dict(k=None), INVALID), (dict(k=FAKE + 2), INVALID), (dict(ks=_st(1280, 640, 0, 1)), INVALID),
                     (dict(ks=_st(1280, 640, 132, 1)), INVALID), (dict(ks=_st(1280, 640, 128, 2)), INVALID), (dict(N=0), INVALID),
                     (dict(start=None), INVALID), (dict(start=FAKE + 1), INVALID), (dict(count=FAKE + 2), INVALID),
                     (dict(theta=0.0), INVALID), (dict(theta=float("nan")), INVALID), (dict(mode=2), UNSUPPORTED),
                     (dict(mode=0x101), UNSUPPORTED), (dict(N=1 << 30), UNSUPPORTED)):
        assert _append(lib, c, **kw) == want, kw
    assert lib.attnfuse_paged_gather(ctypes.byref(c), None, None, FAKE, X, None, X, 5, None) == INVALID
    assert lib.attnfuse_paged_gather(ctypes.byref(c), FAKE + 1, None, FAKE, X, FAKE, X, 5, None) == INVALID
    assert lib.attnfuse_paged_gather(ctypes.byref(c), None, None, FAKE, X, FAKE, X, -1, None) == INVALID


def test_decode_arguments_are_checked(lib):
    c = _cache()
    for kw, want in ((dict(q=None), INVALID), (dict(qs=_st(8 * 128, 132, 1)), INVALID), (dict(lens=None), INVALID),
                     (dict(out=None), INVALID), (dict(out=FAKE + 1), INVALID), (dict(Hq=7), UNSUPPORTED), (dict(Hq=0), INVALID),
                     (dict(scale=0.0), INVALID), (dict(scale=float("inf")), INVALID), (dict(theta=-1.0), INVALID),
                     (dict(mode=2), UNSUPPORTED), (dict(window=-1), INVALID), (dict(slopes=FAKE + 2), INVALID)):
        assert _decode(lib, c, **kw) == want, kw
    n = ctypes.c_size_t()
    for args, want in (((8, 2, 128, 0), OK), ((8, 2, 64, 1), OK), ((8, 3, 128, 0), UNSUPPORTED), ((8, 2, 96, 0), UNSUPPORTED),
                       ((0, 2, 128, 0), INVALID), ((8, 2, 128, 2), INVALID)):
        assert lib.attnfuse_paged_decode_workspace_size(*args, ctypes.byref(n)) == want
    assert lib.attnfuse_paged_decode_workspace_size(8, 2, 128, 0, None) == INVALID
    assert lib.attnfuse_paged_decode_workspace_size(8, 2, 128, 0, ctypes.byref(n)) == OK
    if n.value:
        assert _decode(lib, c, ws=None, ws_n=0) == WS_SMALL
        assert _decode(lib, c, ws_n=n.value - 1) == WS_SMALL
        assert _decode(lib, c, ws=FAKE + 8) == WS_SMALL


def test_binding_refuses_cpu_tensors_and_types():
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="cache k: on cpu"):
        af.PagedCache(pool, pool, table)
    with pytest.raises(TypeError, match="cache k: dtype"):
        af.PagedCache(pool.half(), pool, table)
    with pytest.raises(ValueError, match=r"expected \[num_pages, Hkv, page_size, d\]"):
        af.PagedCache(pool[0], pool, table)
    with pytest.raises(TypeError, match="cache k: expected a torch.Tensor"):
        af.PagedCache(None, pool, table)
    with pytest.raises(TypeError, match="expected a PagedCache"):
        af.paged_decode(pool[:, 0], pool, table)


def test_one_element_dimensions_take_any_stride():
    x = torch.zeros(3, 4, 8, 16)
    assert list(af._live_strides(x)) == list(x.stride())
    odd = torch.as_strided(x, (3, 1, 1, 16), (16, 1, 1, 1))
    assert list(af._live_strides(odd)) == [16, 16, 16, 1]
    assert list(af._live_strides(torch.as_strided(x, (1, 4, 8, 16), (0, 128, 16, 1)))) == [512, 128, 16, 1]
    wide = x.transpose(1, 2)[:, :1]  # slots one, heads behind each other
    assert list(af._live_strides(wide)) == [512, 512, 128, 1]


@pytest.mark.parametrize("d", [64, 128])
def test_row_format(d):
    """Every element has a nibble of its own, and packing is undone by unpacking."""
    at = P.row_nibbles(16, d)
    assert all(sorted(r.tolist()) == list(range(d)) for r in at)
    assert at[0, :4].tolist() == [0, 1, 2, 3] and at[0, 32].item() == 4
    codes = torch.randint(-7, 8, (2, 3, 32, d))
    assert torch.equal(P.unpacked(P.packed(codes)), codes)


def test_reference_quantiser_on_known_groups():
    x = torch.zeros(3, 64).bfloat16()
    x[0, :5] = torch.tensor([7.0, 3.5, -3.5, 0.49, -0.5]).bfloat16()  # step 1: ties away from zero
    x[1, 0] = 2.0 ** -97
    x[2, 40] = float("inf")
    codes, steps = P.quantised(x)
    assert codes[0, :5].tolist() == [7, 4, -4, 0, -1] and steps[0, 0] == 1
    assert steps[1, 0] == 0 and codes[1].abs().sum() == 0
    assert torch.isnan(steps[2, 1]) and steps[2, 0] == 0


def test_more_kv_heads_than_a_grid_holds_are_refused(lib):
    """Heads are a grid dimension of the append and the gather."""
    for q4 in (False, True):
        c = _cache(q4, Hkv=4097)
        assert _append(lib, c) == UNSUPPORTED
        assert lib.attnfuse_paged_gather(ctypes.byref(c), None, None, FAKE, X, FAKE, X, 5, None) == UNSUPPORTED
        assert _decode(lib, c, Hq=4097) == UNSUPPORTED
