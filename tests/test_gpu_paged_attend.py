"""GPU parity: attention of a chunk of new tokens over a paged cache (bf16 and 4-bit) against a
plain 64-bit statement, at the sizes, masks and calls where it can go wrong."""
import math
import random

import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af
from tests import _chunks as K
from tests import _paged as P
from tests.test_gpu_paged import i32, make_cache, randn, table_for

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
DEV = torch.device("cuda")
PAGE_RANGE = 7


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    af.load()
    assert af.device_status() == 0


def run(q, cache, start, count, theta=None, **kw):
    got = af.paged_attend(q, cache, i32(start), None if count is None else i32(count), rope_theta=theta or 1e4,
                          rope_mode=af.ROPE_FUSED if theta else af.ROPE_NONE, **kw)
    torch.cuda.synchronize()
    assert af.device_status() == 0
    return got


def check(q, cache, start, count, theta=None, window=0, slopes=None, scale=None, **kw):
    got = run(q, cache, start, count, theta, window=window, alibi_slopes=slopes, scale=scale, **kw)
    ref = K.attend(q, cache, start, [q.shape[2]] * len(start) if count is None else count,
                   q.shape[-1] ** -0.5 if scale is None else scale, theta, window, slopes)
    K.check(got, ref)
    return got


def slopes_of(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device=DEV)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("d,page", [(128, 16), (64, 48), (128, 80), (64, 256)])
@pytest.mark.parametrize("N", [1, 2, 17, 130])
@pytest.mark.parametrize("theta", [None, 5e5])
def test_lengths_and_pages(q4, d, page, N, theta):
    start = [0, 0, 1, 127, 128, 500, page - 1, 1000]
    count = [N, 0, N, 1, N, max(0, N - 1), N // 2, N]
    cache = make_cache([max(1, s + n) for s, n in zip(start, count)], 2, page, d, q4, seed=N + page)
    check(randn(8, 8, N, d, seed=N), cache, start, count, theta)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (7, 1), (12, 12), (20, 1), (128, 1), (200, 1), (516, 2), (24, 8)])
def test_head_groups(q4, d, Hq, Hkv):
    N = 9
    start, count = [0, 300, 77], [N, N, 5]
    cache = make_cache([s + N for s in start], Hkv, 16, d, q4, seed=Hq)
    check(randn(3, Hq, N, d, seed=Hq), cache, start, count, 1e4)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("N,at", [(1, 40000), (3, 20001), (600, 1500), (1025, 0), (64, 64), (255, 129), (129, 5000)])
def test_one_sequence(q4, N, at):
    cache = make_cache([at + N], 2, 64, 128, q4, seed=N)
    check(randn(1, 8, N, 128, seed=N), cache, [at], None, 5e5)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 1000, 1 << 30])
@pytest.mark.parametrize("alibi", [False, True])
def test_window_and_alibi(q4, window, alibi):
    N, d = 140, 64
    start, count = [0, 900, 128, 2000, 3], [N, 131, N, 0, 1]
    cache = make_cache([max(1, s + n) for s, n in zip(start, count)], 3, 48, d, q4, seed=window % 97)
    check(randn(5, 6, N, d, seed=3), cache, start, count, None, window=window, slopes=slopes_of(6) if alibi else None)


@pytest.mark.parametrize("q4", [False, True])
def test_pages_before_the_window_may_be_gone(q4):
    """Their table entries are not read, and the rows in the window's first page before it may hold anything."""
    N, W, at, page = 20, 200, 1000, 16
    cache = make_cache([at + N], 2, page, 128, q4, seed=5)
    q = randn(1, 8, N, 128, seed=6)
    want = run(q, cache, [at], None, 1e4, window=W)
    first = at - W + 1
    cache.page_table[0, : first // page] = -1
    for pool in (cache.k_scales, cache.v_scales) if q4 else (cache.k, cache.v):
        pool[cache.page_table[0, first // page].item(), :, : first % page] = math.nan
    got = run(q, cache, [at], None, 1e4, window=W)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("q4", [False, True])
def test_large_ragged_batch(q4):
    r = random.Random(8)
    B, N = 40, 300
    start = [r.choice([0, r.randint(0, 3000)]) for _ in range(B)]
    count = [r.choice([0, 1, 1, r.randint(1, N), N]) for _ in range(B)]
    cache = make_cache([max(1, s + n) for s, n in zip(start, count)], 4, 64, 128, q4, seed=9)
    check(randn(B, 16, N, 128, seed=10), cache, start, count, 5e5)


@pytest.mark.parametrize("q4", [False, True])
def test_long_chunks(q4):
    """Units of many tiles, cut and joined."""
    N = 1100
    start, count = [3000, 0, 700], [N, 1000, 33]
    cache = make_cache([s + n for s, n in zip(start, count)], 1, 64, 128, q4, seed=11)
    check(randn(3, 8, N, 128, seed=12), cache, start, count, None)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_uneven_size(q4, d):
    """Elements of sizes e^(2z); scores that grow along the sequence, so that maxima keep moving."""
    N, L = 70, 700
    cache = make_cache([L], 2, 16, d, q4, seed=13, garbage=False)
    g = torch.Generator(DEV).manual_seed(14)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    k = rand(1, 2, L, d) * torch.exp(2 * rand(1, 2, L, 1)) * (1 + torch.arange(L, device=DEV) / 50)[:, None]
    v = rand(1, 2, L, d) * torch.exp(2 * rand(1, 2, L, d))
    af.paged_append(cache, k.bfloat16(), v.bfloat16(), i32([0]), rope_mode=af.ROPE_NONE)
    check(randn(1, 8, N, d, seed=15), cache, [L - N], None, None)
    check(randn(1, 8, N, d, seed=16), cache, [L - N], None, 1e4, window=33)


@pytest.mark.parametrize("q4", [False, True])
def test_sizes_from_tiny_to_large(q4):
    for q_size, k_size, v_size in ((2.0 ** 40, 2.0 ** -38, 2.0 ** 60), (2.0 ** -50, 2.0 ** 52, 2.0 ** -60), (1.0, 1.0, 0.0), (0.0, 1.0, 1.0)):
        cache = make_cache([300], 2, 16, 128, q4, seed=17, garbage=False)
        af.paged_append(cache, randn(1, 2, 300, 128, seed=18) * k_size, randn(1, 2, 300, 128, seed=19) * v_size, i32([0]),
                        rope_mode=af.ROPE_NONE)
        check(randn(1, 8, 50, 128, seed=20) * q_size, cache, [250], None, None)
        check(randn(1, 8, 50, 128, seed=20) * q_size, cache, [250], None, 1e4)


@pytest.mark.parametrize("q4", [False, True])
def test_scores_of_any_size(q4):
    """Scores of some hundreds either way, and a scale of its own."""
    cache = make_cache([400], 1, 16, 128, q4, seed=21)
    check(randn(1, 4, 60, 128, seed=22) * 30, cache, [340], None, None)
    check(-randn(1, 4, 60, 128, seed=22).abs(), cache, [340], None, None, scale=2.0)
    check(randn(1, 4, 60, 128, seed=22), cache, [340], None, 1e4, scale=0.001)


@pytest.mark.parametrize("q4", [False, True])
def test_nan_in_a_visible_row_shows(q4):
    N = 40
    cache = make_cache([200 + N], 1, 16, 128, q4, seed=23, garbage=False)
    (cache.k_scales if q4 else cache.k)[cache.page_table[0, 3].item(), 0, 5] = math.nan
    out, lse = run(randn(1, 4, N, 128, seed=24), cache, [200], None)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("q4", [False, True])
def test_strides_outputs_and_workspace(q4):
    B, Hq, Hkv, N, d = 3, 12, 4, 37, 128
    start, count = [5, 100, 31], [N, 20, N]
    cache = make_cache([s + n for s, n in zip(start, count)], Hkv, 16, d, q4, seed=25)
    q = randn(B, N, Hq + 2, d, seed=26)[:, :, 1:-1].transpose(1, 2)
    want = check(q, cache, start, count, 1e4)
    out = torch.full((B, N, Hq, d + 8), 7.0, device=DEV).bfloat16()
    view = out[..., :d].transpose(1, 2)
    lse = torch.empty(B, Hq, N, device=DEV)
    n = af.paged_attend_workspace_size(B, Hq, Hkv, N, d, cache.format)
    ws = torch.empty(n + 64, dtype=torch.uint8, device=DEV).fill_(0xFF)
    got = run(q, cache, start, count, 1e4, out=view, lse=lse, workspace=ws)
    assert got[0] is view and got[1] is lse
    assert torch.equal(view, want[0]) and torch.equal(lse, want[1]) and (out[..., d:] == 7).all()
    assert (ws[n:] == 0xFF).all()
    none, no_lse = run(q, cache, start, count, 1e4, with_lse=False)
    assert no_lse is None and torch.equal(none, want[0])


@pytest.mark.parametrize("q4", [False, True])
def test_strided_pools(q4):
    start, N, page, d = [40, 7], 30, 16, 128
    a = make_cache([s + N for s in start], 3, page, d, q4, seed=27)
    row = d // 2 if q4 else d

    def spread(x, heads, pad):
        if x is None:
            return None
        big = torch.zeros(x.shape[0], heads, page, x.shape[3] + pad, dtype=x.dtype, device=DEV)
        view = big[:, 1:1 + x.shape[1], :, : x.shape[3]]
        view.copy_(x)
        return view

    pad = 0 if q4 else 8
    b = af.PagedCache(spread(a.k, 5, pad), spread(a.v, 6, pad), a.page_table, spread(a.k_scales, 5, 0), spread(a.v_scales, 7, 0))
    assert row and not b.k.is_contiguous()
    q = randn(2, 6, N, d, seed=28)
    want, got = run(q, a, start, None, 1e4), run(q, b, start, None, 1e4)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("q4", [False, True])
def test_offsets_past_32_bits(q4):
    """A pool whose last pages lie more than 2^32 bytes behind its first."""
    page, d, Hkv, N = 16, 128, 2, 40
    bytes_row = d // 2 if q4 else 2 * d
    P_ = (1 << 32) // (Hkv * page * bytes_row) + 40
    small = make_cache([300 + N], Hkv, page, d, q4, seed=29)
    new = lambda x: torch.zeros(P_, *x.shape[1:], dtype=x.dtype, device=DEV) if x is not None else None  # noqa: E731
    pools = [new(x) for x in (small.k, small.v, small.k_scales, small.v_scales)]
    table = small.page_table.clone()
    for i in range(-(-(300 + N) // page)):
        to = P_ - 1 - i
        for big, x in zip(pools, (small.k, small.v, small.k_scales, small.v_scales)):
            if big is not None:
                big[to] = x[table[0, i].item()]
        table[0, i] = to
    big = af.PagedCache(pools[0], pools[1], table, pools[2], pools[3])
    q = randn(1, 8, N, d, seed=30)
    want, got = run(q, small, [300], None, 1e4), run(q, big, [300], None, 1e4)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("q4", [False, True])
def test_bad_pages_starts_and_counts_are_skipped_and_reported(q4):
    N, page, d, Hkv = 40, 16, 128, 2
    start, count = [200, 0, 90, 300], [N, 17, N, 8]
    cache = make_cache([s + n for s, n in zip(start, count)], Hkv, page, d, q4, seed=31)
    q = randn(4, 8, N, d, seed=32)
    good = run(q, cache, start, count, 1e4)

    def call(start, count, table=None):
        c = cache if table is None else af.PagedCache(cache.k, cache.v, table, cache.k_scales, cache.v_scales)
        got = af.paged_attend(q, c, i32(start), i32(count), rope_theta=1e4)
        torch.cuda.synchronize()
        assert af.device_status() == PAGE_RANGE
        assert af.device_status() == 0
        return got

    def same(got, want, rows):
        return all(torch.equal(a[b], w[b]) for a, w in zip(got, want) for b in rows)

    # a page behind the pool: its 16 keys are as if they were not there
    for bad in (-1, cache.num_pages, 1 << 30, -(1 << 31)):
        table = cache.page_table.clone()
        table[0, 3] = bad
        got = call(start, count, table)
        assert same(got, good, (1, 2, 3))
        keep = [i for i in range(240) if not 48 <= i < 64]
        k, v = (P.rows(P.values(cache, n), cache.page_table, 0, 0, 240)[:, keep] for n in "kv")
        pos = torch.arange(200, 240, device=DEV)
        qr = P.rotated(q[0].double(), pos, 1e4).view(Hkv, 4, N, d)
        x = torch.einsum("hgic,hnc->hgin", qr, k) * d ** -0.5
        x = x.masked_fill(torch.tensor(keep, device=DEV) > pos[:, None], -math.inf)
        o = torch.einsum("hgin,hnc->hgic", torch.softmax(x, -1), v)
        assert (got[0][0].double() - o.view(8, N, d)).abs().max() <= 2.0 ** -5
        assert (got[1][0].double() - torch.logsumexp(x, -1).view(8, N)).abs().max() <= 2.0 ** -9
    # counts outside [0, N] are clamped
    got = call(start, [N, -3, N, 8])
    assert same(got, good, (0, 2, 3)) and (got[0][1] == 0).all() and (got[1][1] == -math.inf).all()
    got = call(start, [N + 100, 17, N, 8])
    assert same(got, good, (0, 1, 2, 3))
    # starts outside the table: rows without a position are padding
    cap = cache.max_pages * page
    for s in (-1, -(1 << 31), cap, (1 << 31) - 1):
        got = call([200, 0, 90, s], count)
        assert same(got, good, (0, 1, 2)) and (got[0][3] == 0).all() and (got[1][3] == -math.inf).all()


@pytest.mark.parametrize("q4", [False, True])
def test_captured_calls_follow_the_device_values(q4):
    B, Hq, Hkv, N, d, page = 3, 8, 2, 33, 128, 16
    caches = [make_cache([500 + N] * B, Hkv, page, d, q4, seed=33 + i) for i in range(2)]
    cache = caches[0]
    q, start, count = randn(B, Hq, N, d, seed=35), i32([0, 5, 400]), i32([N, 1, 7])
    out, lse = torch.empty_like(q), torch.empty(B, Hq, N, device=DEV)
    ws = [torch.empty(af.paged_attend_workspace_size(B, Hq, Hkv, N, d, cache.format), dtype=torch.uint8, device=DEV) for _ in range(2)]
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    af.paged_attend(q, cache, start, count, out=out, lse=lse, workspace=ws[0])
    torch.cuda.synchronize()
    for g, o, l, w in zip(graphs, (out, out2), (lse, lse2), ws):
        with torch.cuda.graph(g):
            af.paged_attend(q, cache, start, count, out=o, lse=l, workspace=w)
    for s, c in (([0, 5, 400], [N, 1, 7]), ([499, 0, 3], [0, N, N]), ([500, 500, 500], [N, N, N]), ([1, 2, 3], [0, 0, 0])):
        start.copy_(i32(s)), count.copy_(i32(c))
        q.copy_(randn(B, Hq, N, d, seed=sum(s)))
        streams = [torch.cuda.Stream() for _ in range(2)]
        for g, st in zip(graphs, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        ref = K.attend(q, cache, s, c, d ** -0.5, 1e4)
        K.check((out, lse), ref)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert af.device_status() == 0


@pytest.mark.parametrize("q4", [False, True])
def test_calls_on_two_streams_at_once_and_results_do_not_vary(q4):
    B, N = 6, 150
    start = [0, 900, 2000, 17, 1500, 64]
    cache = make_cache([s + N for s in start], 2, 64, 128, q4, seed=36)
    q = randn(B, 16, N, 128, seed=37)
    want = run(q, cache, start, None, 5e5)
    streams = [torch.cuda.Stream() for _ in range(3)]
    first = i32(start)
    torch.cuda.synchronize()
    got = [af.paged_attend(q, cache, first, rope_theta=5e5, stream=s) for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


@pytest.mark.parametrize("q4", [False, True])
def test_a_row_does_not_depend_on_the_heads_and_rows_beside_it_in_value(q4):
    """One token alone, through the attention of chunks and through the decode."""
    B, Hq, Hkv, d = 5, 8, 2, 128
    lens = [1, 100, 129, 1000, 2500]
    cache = make_cache(lens, Hkv, 16, d, q4, seed=38)
    q = randn(B, Hq, 1, d, seed=39)
    out, lse = check(q, cache, [n - 1 for n in lens], None, 5e5)
    ref, ref_lse = af.paged_decode(q[:, :, 0], cache, i32(lens), rope_theta=5e5)
    # both are within their own tolerances of the exact value, of at most 2^-6 of values near 1
    assert (out[:, :, 0].float() - ref.float()).abs().max() <= 2.0 ** -5
    assert (lse[:, :, 0] - ref_lse).abs().max() <= 2.0 ** -9


@pytest.mark.parametrize("q4", [False, True])
def test_rotation_append_attention_and_decode_together(q4):
    """Two chunks of prompts with positions on three axes, then single tokens."""
    B, Hq, Hkv, d, page = 3, 8, 2, 128, 16
    sections = (16, 24, 24)
    total = 90
    table, n = table_for([total + 4] * B, page, 40)
    cache = af.PagedCache.empty(n, Hkv, page, d, table, q4=q4)
    q, k, v = (randn(B, h, total, d, seed=41 + i) for i, h in enumerate((Hq, Hkv, Hkv)))
    pos = torch.randint(0, 400, (3, B, total), generator=torch.Generator(DEV).manual_seed(44), device=DEV, dtype=torch.int32)
    rows = []
    for a, b in ((0, 61), (61, 89), (89, 90)):
        rq, rk = af.rope_axes(q[:, :, a:b], k[:, :, a:b], pos[:, :, a:b], sections)
        af.paged_append(cache, rk, v[:, :, a:b], i32([a] * B), rope_mode=af.ROPE_NONE)
        if b - a > 1:
            rows.append(run(rq, cache, [a] * B, None))
        else:
            o, l = af.paged_decode(rq[:, :, 0].contiguous(), cache, i32([b] * B), rope_mode=af.ROPE_NONE)
            rows.append((o[:, :, None], l[:, :, None]))
    got = [torch.cat(x, 2) for x in zip(*rows)]
    rq, rk = af.rope_axes(q, k, pos, sections)
    if not q4:
        want, want_lse = af.fwd(rq, rk, v, rope_mode=af.ROPE_NONE, variant=af.Variant(mask=af.MASK_CAUSAL))
        assert (got[0].float() - want.float()).abs().max() <= 2.0 ** -5 and (got[1] - want_lse).abs().max() <= 2.0 ** -9
    K.check(got, K.attend(rq, cache, [0] * B, [total] * B, d ** -0.5))


@pytest.mark.parametrize("seed", range(40))
def test_random_calls(seed):
    """Sizes, groups, pages, windows, bias and rotation of any mix."""
    r = random.Random(1000 + seed)
    d, q4 = r.choice([64, 128]), r.random() < 0.5
    Hkv, g = r.choice([1, 2, 3, 5]), r.choice([1, 2, 3, 4, 5, 8, 11, 16, 33])
    B, N, page = r.randint(1, 9), r.choice([1, 2, 7, 40, 129, 260, 400]), r.choice([16, 32, 48, 64, 112, 128, 256, 400])
    start = [r.choice([0, r.randint(0, 200), r.randint(0, 1500)]) for _ in range(B)]
    count = [r.choice([0, 1, N, r.randint(0, N)]) for _ in range(B)]
    cache = make_cache([max(1, s + n) for s, n in zip(start, count)], Hkv, page, d, q4, seed=seed)
    check(randn(B, Hkv * g, N, d, seed=seed), cache, start, count, r.choice([None, 1e4]),
          window=r.choice([0, 0, 1, r.randint(2, 400)]), slopes=slopes_of(Hkv * g) if r.random() < 0.3 else None)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("window", [1, 100, 1000])
def test_positions_up_to_the_last(q4, window):
    """A table of 2^24 positions over a few pages that it names again and again."""
    N, page, end = 40, 256, 1 << 24
    small = make_cache([4 * page], 2, page, 64, q4, seed=70, garbage=False)
    table = (torch.arange(end // page, device=DEV, dtype=torch.int32) % 4)[None].contiguous()
    cache = af.PagedCache(small.k, small.v, table, small.k_scales, small.v_scales)
    check(randn(1, 4, N, 64, seed=71), cache, [end - N], None, 5e5, window=window)


@pytest.mark.parametrize("q4", [False, True])
def test_the_largest_group(q4):
    cache = make_cache([40, 200], 1, 16, 64, q4, seed=60)
    check(randn(2, 4096, 2, 64, seed=61), cache, [38, 198], [2, 1], 1e4)


@pytest.mark.parametrize("q4", [False, True])
def test_many_short_sequences(q4):
    """More of them than threads and CTAs, most without new tokens."""
    r = random.Random(62)
    B = 1500
    start = [r.randint(0, 60) for _ in range(B)]
    count = [r.choice([0, 0, 0, 1, 2, 3]) for _ in range(B)]
    cache = make_cache([max(1, s + n) for s, n in zip(start, count)], 1, 16, 64, q4, seed=63)
    check(randn(B, 2, 3, 64, seed=64), cache, start, count, 1e4)
    check(randn(B, 2, 3, 64, seed=65), cache, start, [0] * B, 1e4)


@pytest.mark.parametrize("q4", [False, True])
def test_a_key_of_large_values_that_others_see_last(q4):
    """A chunk's last key and value are 2^20 times the others: rows before it keep their bits."""
    N = 50
    cache = make_cache([300 + N], 2, 16, 128, q4, seed=66, garbage=False)
    q = randn(1, 8, N, 128, seed=67)
    k, v = randn(1, 2, 1, 128, seed=68) * 2.0 ** 20, randn(1, 2, 1, 128, seed=69) * 2.0 ** 20
    af.paged_append(cache, k, v, i32([300 + N - 1]), rope_mode=af.ROPE_NONE)
    out, lse = run(q, cache, [300], None)
    ref = K.attend(q, cache, [300], [N], 128 ** -0.5)
    K.check((out[:, :, :-1].contiguous(), lse[:, :, :-1].contiguous()), [x[:, :, :-1] for x in ref])


@pytest.mark.parametrize("q4", [False, True])
def test_shared_pages(q4):
    """Sequences that share a prompt's pages."""
    cache = make_cache([320], 2, 16, 128, q4, seed=45)
    table = cache.page_table.expand(4, -1).contiguous()
    c = af.PagedCache(cache.k, cache.v, table, cache.k_scales, cache.v_scales)
    check(randn(4, 8, 20, 128, seed=46), c, [300, 100, 0, 250], [20, 20, 20, 1], 1e4)


def test_refusals_on_the_gpu():
    cache = make_cache([64, 64], 2, 16, 64, False, seed=47)
    q, start = randn(2, 4, 8, 64, seed=48), i32([0, 0])
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(q=q[:, :3]), dict(q=q.cpu()), dict(q=q[..., :32]), dict(start=None), dict(start=start.long()),
                dict(start=start[:1]), dict(start=start.cpu()), dict(count=start.float()), dict(out=q.float()), dict(out=q[:, :2]),
                dict(lse=torch.empty(2, 4, 7, device=DEV)), dict(lse=torch.empty(2, 8, 4, device=DEV).transpose(1, 2)), dict(window=-1),
                dict(window=-(1 << 40)), dict(alibi_slopes=torch.ones(3, device=DEV)), dict(scale=0.0), dict(scale=math.nan),
                dict(rope_mode=af.ROPE_PREROTATE), dict(rope_theta=-1.0), dict(workspace=torch.empty(1 << 20)), dict(q=q[:, :, :0]),
                dict(cache=cache.k)):
        args = dict(q=q, cache=cache, start=start) | bad
        with pytest.raises((ValueError, TypeError, af.AttnfuseError)):
            af.paged_attend(**args)
    assert af.device_status() == 0
