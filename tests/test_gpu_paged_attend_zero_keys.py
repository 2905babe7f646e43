"""GPU parity: attention of chunks where keys, queries or both are zero or tiny. A row without a
score takes the mean of the values that it sees, and its lse is the logarithm of their number."""
import math

import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af
from tests import _chunks as K
from tests.test_gpu_paged import i32, make_cache, randn, table_for
from tests.test_gpu_paged_attend import PAGE_RANGE, check, run, slopes_of

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
DEV = torch.device("cuda")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    af.load()
    assert af.device_status() == 0


def cache_of(lens, Hkv, d, q4, k_size, seed):
    """Keys of the given size, values near 1."""
    L = max(lens)
    cache = make_cache([L] * len(lens), Hkv, 16, d, q4, seed=seed, garbage=False)
    k, v = (randn(len(lens), Hkv, L, d, seed=seed + i) for i in (1, 2))
    af.paged_append(cache, k * k_size, v, i32([0] * len(lens)), rope_mode=af.ROPE_NONE)
    return cache


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 5, 60])  # with groups of 4, a row tile and two
@pytest.mark.parametrize("theta", [None, 1e4])
@pytest.mark.parametrize("k_size", [0.0, 2.0 ** -99, 2.0 ** -90, 2.0 ** -40, 1.0])
def test_small_queries_and_keys(q4, d, N, theta, k_size):
    start, count = [0, 1, 127, 300, 200], [N, N, N, max(1, N - 3), 0]
    cache = cache_of([s + N for s in start], 2, d, q4, k_size, seed=N)
    q = randn(5, 8, N, d, seed=N + 9)
    for q_size in (0.0, 2.0 ** -126, 2.0 ** -100, 2.0 ** -40, 2.0 ** -9, 1.0):
        for window, slopes in ((0, None), (33, None), (0, slopes_of(8))):
            check(q * q_size, cache, start, count, theta, window=window, slopes=slopes)


@pytest.mark.parametrize("q4", [False, True])
def test_zero_rows_among_others(q4):
    """Padding tokens: the first keys of a sequence and some queries are zero, and no others."""
    N = 70
    cache = make_cache([500, 500], 2, 16, 128, q4, seed=3, garbage=False)
    k, v = randn(2, 2, 500, 128, seed=4), randn(2, 2, 500, 128, seed=5)
    k[:, :, :200] = 0
    af.paged_append(cache, k, v, i32([0, 0]), rope_mode=af.ROPE_NONE)
    q = randn(2, 8, N, 128, seed=6)
    q[:, :, ::3] = 0
    for start in ([0, 430], [100, 190], [64, 128]):
        for theta in (None, 1e4):
            check(q, cache, start, None, theta)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("N", [1, 8, 100])
def test_a_call_on_zeros_alone(q4, N):
    """A warm-up or a capture on buffers of zeros."""
    start = [0, 40, 128]
    table, n = table_for([s + N for s in start], 16, 7)
    cache = af.PagedCache.empty(n, 2, 16, 128, table, q4=q4)
    for pool in (cache.k, cache.v, cache.k_scales, cache.v_scales):
        if pool is not None:
            pool.zero_()
    out, lse = run(torch.zeros(3, 8, N, 128, device=DEV).bfloat16(), cache, start, None, 1e4)
    assert (out == 0).all()
    want = torch.log(torch.tensor(start, device=DEV).double()[:, None, None] + 1 + torch.arange(N, device=DEV))
    assert ((lse.double() - want).abs() <= 2.0 ** -20 * (1 + want)).all()
    last = i32([s + 1 for s in start])
    out, lse = af.paged_decode(torch.zeros(3, 8, 128, device=DEV).bfloat16(), cache, last, rope_theta=1e4)
    assert (out == 0).all()
    assert ((lse.double() - want[:, :, 0]).abs() <= 2.0 ** -20 * (1 + want[:, :, 0])).all()


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("N", [5, 60])
def test_a_tile_without_a_page(q4, N):
    """No page of a whole key tile is one (the first, the one in the middle, the last): small queries
    see the others, or none."""
    at, page, d = 384, 16, 128
    cache = cache_of([at], 2, d, q4, 1.0, seed=8)
    q = randn(1, 8, N, d, seed=9) * 2.0 ** -12
    tile = 128 // page
    for gone in ((0,), (1,), (2,), (0, 1, 2)):
        table = cache.page_table.clone()
        for t in gone:
            table[0, t * tile: (t + 1) * tile] = -1
        c = af.PagedCache(cache.k, cache.v, table, cache.k_scales, cache.v_scales)
        out, lse = af.paged_attend(q, c, i32([at - N]), rope_mode=af.ROPE_NONE)
        torch.cuda.synchronize()
        assert af.device_status() == PAGE_RANGE
        keep = [i for i in range(at) if i // 128 not in gone]
        if not keep:
            assert (out == 0).all() and (lse == -math.inf).all()
            continue
        # the keys that are left as a sequence of their own, its rows behind all of them or as far into the last tile
        hidden = 128 * len([t for t in gone if t < 2])
        if 2 in gone:
            # every row sees all 256 of the first two tiles: as if it stood at the last of them
            ref = K.attend(q.transpose(0, 2).contiguous(), _first(cache, 256, N), [255] * N, [1] * N, d ** -0.5)
            ref = [x.transpose(0, 2) for x in ref]
        else:
            left = [p for t in range(3) if t not in gone for p in cache.page_table[0, t * tile: (t + 1) * tile].tolist()]
            short = af.PagedCache(cache.k, cache.v, i32([left]), cache.k_scales, cache.v_scales)
            ref = K.attend(q, short, [at - N - hidden], [N], d ** -0.5)
        K.check((out, lse), ref)


def _first(cache, n, B):
    """The first n positions of a cache's only sequence, for B sequences."""
    table = cache.page_table[:, : n // cache.page_size].expand(B, -1).contiguous()
    return af.PagedCache(cache.k, cache.v, table, cache.k_scales, cache.v_scales)


@pytest.mark.parametrize("q4", [False, True])
def test_scales_below_the_normal_range(q4):
    """A scale of 2^-130 over products of some 2^125: scores of some 2^-5."""
    cache = cache_of([300], 2, 64, q4, 2.0 ** 61, seed=10)
    check(randn(1, 8, 50, 64, seed=13).clamp(-3, 3) * 2.0 ** 61, cache, [250], None, None, scale=2.0 ** -130)
