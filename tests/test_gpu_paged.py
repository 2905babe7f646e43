"""GPU parity: paged caches (append, gather, decode; bf16 and 4-bit) against plain 64-bit
statements of the same operators, at the sizes and masks where they can go wrong."""
import math
import random

import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af
from tests import _paged as P

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


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def table_for(lens, page, seed, spare=3, wide=1):
    """(page_table with pages in random order and garbage behind each sequence's, num_pages)."""
    r = random.Random(seed)
    need = [-(-n // page) for n in lens]
    pages = list(range(sum(need) + spare))
    r.shuffle(pages)
    width = max(need) + wide
    rows = []
    for n in need:
        rows.append([pages.pop() for _ in range(n)] + [r.choice([-1, 1 << 30, -(1 << 31)]) for _ in range(width - n)])
    return i32(rows), sum(need) + spare


def make_cache(lens, Hkv, page, d, q4, seed, garbage=True):
    """A cache whose sequences hold lens[b] random rows; every other slot holds NaN (bf16: values,
    q4: steps), as memory that nothing has written yet may."""
    g = torch.Generator(DEV).manual_seed(seed)
    table, n = table_for(lens, page, seed)
    live = torch.zeros(n, page, dtype=torch.bool, device=DEV)
    for b, L in enumerate(lens):
        p = torch.arange(L, device=DEV)
        live[table[b, p // page].long(), p % page] = True
    live = live[:, None, :, None] | (not garbage)
    pools = []
    for _ in "kv":
        x = torch.randn(n, Hkv, page, d, generator=g, device=DEV)
        if q4:
            codes, steps = P.quantised(x.bfloat16())
            pools.append((P.packed(codes), torch.where(live, steps, torch.full_like(steps, math.nan))))
        else:
            pools.append((torch.where(live, x, torch.full_like(x, math.nan)).bfloat16(), None))
    (k, ks), (v, vs) = pools
    return af.PagedCache(k, v, table, ks, vs)


def randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator(DEV).manual_seed(seed), device=DEV).bfloat16()


# ---------------------------------------------------------------------------------------------
# append and gather
# ---------------------------------------------------------------------------------------------
def expected_append(cache, k, v, start, count, theta):
    """The pools after an append, from copies taken before it."""
    want = {n: getattr(cache, n).clone() for n in ("k", "v")}
    if cache.q4:
        want |= {n: getattr(cache, n).clone() for n in ("k_scales", "v_scales")}
    S, d = cache.page_size, cache.d
    nib = P.row_nibbles(S, d).to(DEV) if cache.q4 else None
    for b in range(cache.B):
        p = start[b] + torch.arange(count[b], device=DEV)
        page, slot = cache.page_table[b, p // S].long(), p % S
        for n, x in (("k", k), ("v", v)):
            x = x[b, :, :count[b]]
            row = P.as_row(P.rotated(x, p, theta)) if n == "k" and theta else x
            row = row.transpose(0, 1)  # [rows, Hkv, d]
            if not cache.q4:
                want[n][page, :, slot] = row
                continue
            codes, steps = P.quantised(row)
            q = torch.zeros_like(codes).scatter_(2, nib[slot][:, None].expand_as(codes), codes + 8)
            want[n][page, :, slot] = (q[..., 0::2] | (q[..., 1::2] << 4)).to(torch.uint8)
            want[n + "_scales"][page, :, slot] = steps
    return want


def check_append(cache, k, v, start, count, theta, **kw):
    want = expected_append(cache, k, v, start, count, theta)
    mode = af.ROPE_FUSED if theta else af.ROPE_NONE
    af.paged_append(cache, k, v, i32(start), i32(count) if kw.pop("counts", True) else None,
                    rope_theta=theta or 1e4, rope_mode=mode, **kw)
    torch.cuda.synchronize()
    assert af.device_status() == 0
    for n, w in want.items():
        got = getattr(cache, n)
        same = (got == w) | ((got != got) & (w != w))
        assert same.all(), f"{n}: {(~same).sum().item()} of {same.numel()} differ"


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("d,Hkv,page,theta", [(128, 8, 16, 5e5), (128, 2, 48, 1e4), (64, 16, 64, 1e4),
                                              (64, 1, 256, None), (128, 1, 128, None), (128, 12, 80, 5e5)])
@pytest.mark.parametrize("N", [1, 7, 200])
def test_append(q4, d, Hkv, page, theta, N):
    B = 5
    r = random.Random(N * page + d)
    start = [0, 1, page - 1, 3 * page, 1000]
    count = [N, 0, r.randint(0, N), N, N]
    cache = make_cache([s + N for s in start], Hkv, page, d, q4, seed=N)
    k, v = randn(B, Hkv, N, d, seed=1), randn(B, Hkv, N, d, seed=2)
    check_append(cache, k, v, start, count, theta)


@pytest.mark.parametrize("q4", [False, True])
def test_append_many_heads_per_thread(q4):
    """Enough rows that a thread keeps a run of heads, which does not divide Hkv."""
    B, Hkv, N, d = 3, 11, 6001, 128
    cache = make_cache([N + 5] * B, Hkv, 64, d, q4, seed=3, garbage=False)
    check_append(cache, randn(B, Hkv, N, d, seed=4), randn(B, Hkv, N, d, seed=5), [5, 0, 1], [N, 17, N - 1], 5e5)


@pytest.mark.parametrize("q4", [False, True])
def test_append_strided_inputs_and_pools(q4):
    """k, v as views of a fused projection [B, N, H, d], pools as views of a larger allocation
    with another order of heads and pages, no counts."""
    B, Hkv, N, d, page = 2, 4, 33, 64, 32
    qkv = randn(B, N, 3, Hkv, d + 8, seed=6)
    k, v = qkv[:, :, 1, :, 8:].transpose(1, 2), qkv[:, :, 2, :, :d].transpose(1, 2)
    table, n = table_for([N + 9] * B, page, 8)
    if q4:
        big = torch.full((Hkv, n, 2, page, d // 2), 0x88, dtype=torch.uint8, device=DEV)
        sc = torch.zeros(Hkv, n, 2, page, d // 32, dtype=torch.bfloat16, device=DEV)
        kp, vp = big[:, :, 0].transpose(0, 1), big[:, :, 1].transpose(0, 1)
        cache = af.PagedCache(kp, vp, table, sc[:, :, 0].transpose(0, 1), sc[:, :, 1].transpose(0, 1))
    else:
        big = torch.zeros(n, page, 2, Hkv, d, dtype=torch.bfloat16, device=DEV)
        cache = af.PagedCache(big[:, :, 0].transpose(1, 2), big[:, :, 1].transpose(1, 2), table)
    check_append(cache, k, v, [9, 0], [N, N], 1e4, counts=False)


def test_append_rotates_exactly_at_far_positions():
    """Positions up to 2^24 - 1: the fp32 angle with its residual, the fp64 path at borders."""
    B, Hkv, N, d, page = 1, 2, 64, 128, 1 << 14
    top = (1 << 24) - N
    table = torch.full((1, 1 << 10), -1, dtype=torch.int32, device=DEV)
    table[0, -1] = 0
    pool = lambda: torch.zeros(1, Hkv, page, d, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    cache = af.PagedCache(pool(), pool(), table)
    for theta in (1e4, 5e5):
        check_append(cache, randn(B, Hkv, N, d, seed=9), randn(B, Hkv, N, d, seed=10), [top], [N], theta)


def test_row_bits_do_not_depend_on_the_batch():
    """A row written in a prompt has the bits of the same row written alone."""
    Hkv, N, d, page = 8, 100, 128, 16
    for q4 in (False, True):
        a = make_cache([N], Hkv, page, d, q4, seed=11, garbage=False)
        b = af.PagedCache(*[None if x is None else x.clone() for x in (a.k, a.v, a.page_table, a.k_scales, a.v_scales)])
        k, v = randn(1, Hkv, N, d, seed=12), randn(1, Hkv, N, d, seed=13)
        af.paged_append(a, k, v, i32([0]), rope_theta=5e5)
        for n in range(N):
            af.paged_append(b, k[:, :, n:n + 1], v[:, :, n:n + 1], i32([n]), rope_theta=5e5)
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
        if q4:
            assert torch.equal(a.k_scales, b.k_scales) and torch.equal(a.v_scales, b.v_scales)


def test_q4_quantisation_edges():
    """Ties, signs, one-element groups, zeros, tiny and huge groups, infinities and NaN."""
    d, page, Hkv, B = 128, 16, 1, 1
    x = torch.zeros(24, d)
    for i in range(7):  # step exactly 2^e: ties at every k + 1/2, both signs
        e = 2.0 ** (10 * i - 30)
        x[i, :32] = torch.tensor([(j - 15.5) / 2 for j in range(32)]).clamp(-7, 7) * e
        x[i, 0], x[i, 31] = -7 * e, 7 * e
    x[7, ::32] = torch.tensor([1.0, -1.0, 3e-20, -2e30])           # one element per group
    x[8, :32], x[8, 32:64], x[8, 64:96] = 2.0 ** -97, 2.0 ** -96, -2.0 ** -96
    x[9, 3], x[9, 40], x[9, 70] = math.inf, -math.inf, math.nan
    x[10, :] = 3.38e38
    x[11, 5] = -3.38e38
    x[12:] = torch.randn(12, d, generator=torch.Generator().manual_seed(1)) * torch.logspace(-25, 25, d)
    x = x.bfloat16().to(DEV).view(1, 1, 24, d)
    cache = make_cache([24], Hkv, page, d, True, seed=14, garbage=False)
    want = {n: P.quantised(x[0, 0])[i] for i, n in enumerate(("codes", "steps"))}
    af.paged_append(cache, x, x, i32([0]), rope_mode=af.ROPE_NONE)
    k, v = af.paged_gather(cache, None, None, 24)
    torch.cuda.synchronize()
    assert af.device_status() == 0
    val = (want["codes"].double() * want["steps"].double().repeat_interleave(32, -1)).float().bfloat16()
    for got in (k, v):
        got = got[0, 0]
        assert torch.equal(torch.isnan(got), torch.isnan(val))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(val))
    # the format's own promise, from the values alone: at most half a step off, but for the
    # rounding of the step, 7 * 2^-9 of it
    y, s = x[0, 0].double(), want["steps"].double().repeat_interleave(32, -1)
    fine = torch.isfinite(s) & (s > 0) & (y.abs() < 1e38)
    off = (want["codes"].double() * s - y).abs()
    assert (off[fine] <= (0.5 + 7 * 2.0 ** -8) * s[fine]).all()


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 48), (128, 128)])
def test_gather(q4, d, page):
    lens, N, Hkv = [0, 5, 300, 64, 129], 200, 3
    cache = make_cache(lens, Hkv, page, d, q4, seed=15)
    start, count = [0, 2, 37, 0, 128], [0, 3, 200, 64, 1]
    big = torch.full((5, N, Hkv, 2, d), 7.0, dtype=torch.bfloat16, device=DEV)
    k, v = af.paged_gather(cache, i32(start), i32(count), N, k=big[..., 0, :].transpose(1, 2))
    torch.cuda.synchronize()
    assert af.device_status() == 0
    for got, which in ((k, "k"), (v, "v")):
        pool = P.values(cache, which)
        for b in range(5):
            want = P.rows(pool, cache.page_table, b, start[b], count[b]).float().bfloat16()
            assert torch.equal(got[b, :, :count[b]], want)
            assert (got[b, :, count[b]:] == 0).all()
    assert (big[..., 1, :] == 7).all()


# ---------------------------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------------------------
def run_decode(lens, Hq, Hkv, page, d, q4, theta=None, window=0, slopes=None, seed=0, cache=None, **kw):
    cache = cache or make_cache(lens, Hkv, page, d, q4, seed)
    q = randn(len(lens), Hq, d, seed=seed + 50)
    got = af.paged_decode(q, cache, i32(lens), rope_theta=theta or 1e4,
                          rope_mode=af.ROPE_FUSED if theta else af.ROPE_NONE, window=window, alibi_slopes=slopes, **kw)
    torch.cuda.synchronize()
    assert af.device_status() == 0
    P.check_decode(got, P.decode(q, cache, i32(lens), d ** -0.5, theta, window, slopes))
    return got


EDGES = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 191, 193, 255, 257, 511, 1000]


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 48, 64, 80, 256])
def test_decode_lengths_and_pages(q4, d, page):
    run_decode(EDGES, 8, 2, page, d, q4, theta=5e5, seed=page)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (12, 12), (6, 3), (7, 1), (8, 1), (9, 1), (16, 1), (40, 2), (17, 1), (64, 2)])
def test_decode_head_groups(q4, d, Hq, Hkv):
    run_decode([700, 3, 0, 129], Hq, Hkv, 32, d, q4, theta=1e4, seed=Hq)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("L", [1, 64, 65, 4095, 20000])
def test_decode_one_sequence(q4, L):
    """One sequence split over many CTAs."""
    run_decode([L], 8, 1, 64, 128, q4, theta=5e5, seed=L)
    run_decode([L], 16, 1, 64, 64, q4, theta=None, seed=L)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("window", [1, 16, 63, 64, 65, 200, 5000])
def test_decode_window_and_alibi(q4, window):
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / 8) for h in range(8)], device=DEV)
    run_decode(EDGES + [3001], 8, 2, 16, 128, q4, theta=1e4, window=window, slopes=slopes, seed=window)
    run_decode(EDGES + [3001], 8, 8, 64, 64, q4, window=window, seed=window)


@pytest.mark.parametrize("q4", [False, True])
def test_decode_alibi_alone(q4):
    slopes = torch.tensor([0.5, 2.0 ** -8, 0.0, -0.25], device=DEV)
    run_decode([2500, 64, 1, 0], 4, 2, 32, 128, q4, slopes=slopes, seed=3)


@pytest.mark.parametrize("q4", [False, True])
def test_decode_large_ragged_batch(q4):
    """More sequences than CTAs, most of one tile, some long: every kind of run of tiles."""
    r = random.Random(5)
    lens = [r.choice([0, 1, r.randint(1, 64), r.randint(1, 300), r.randint(1, 3000)]) for _ in range(333)]
    run_decode(lens, 4, 2, 16, 64, q4, theta=1e4, seed=5)
    run_decode(lens[:150], 16, 2, 48, 128, q4, theta=1e4, seed=6)


@pytest.mark.parametrize("q4", [False, True])
def test_decode_values_of_uneven_size(q4):
    """Keys that dominate, values and steps over many magnitudes, constant rows: the running
    maximum and the 4-bit weights' exponents move in both directions along a sequence."""
    lens, Hkv, page, d = [900, 900], 2, 32, 128
    cache = make_cache(lens, Hkv, page, d, q4, seed=21, garbage=False)
    g = torch.Generator(DEV).manual_seed(22)
    for which in "kv":
        pool = getattr(cache, which + "_scales") if q4 else getattr(cache, which)
        shape = (pool.shape[0], 1, pool.shape[2], 1)
        lo, hi = (-1.0, 1.5) if which == "k" else (-9.0, 9.0)
        f = torch.exp(lo + (hi - lo) * torch.rand(shape, generator=g, device=DEV))
        if which == "v":  # channels groups of their own size too
            f = f * torch.logspace(-4, 4, pool.shape[3], device=DEV)
        pool.copy_((pool.float() * f).bfloat16())
    run_decode(lens, 8, Hkv, page, d, q4, theta=1e4, seed=23, cache=cache)


def test_decode_zero_and_extreme_values_q4():
    """All-zero values (steps 0) give 0; values at both ends of what a step can hold stay finite."""
    lens, Hkv, page, d = [300, 70], 1, 16, 128
    for f in (0.0, 2.0 ** -96, 1e34):
        cache = make_cache(lens, Hkv, page, d, True, seed=24, garbage=False)
        cache.v_scales.copy_((cache.v_scales.float() * f).bfloat16())
        run_decode(lens, 8, Hkv, page, d, True, theta=1e4, seed=25, cache=cache)


@pytest.mark.parametrize("q4", [False, True])
def test_decode_nan_in_a_visible_row_shows(q4):
    """A NaN inside the length reaches its head's output, and nothing else."""
    lens, Hkv, page, d = [200, 200], 2, 16, 128
    cache = make_cache(lens, Hkv, page, d, q4, seed=26, garbage=False)
    p = cache.page_table[1, 100 // page].item()
    (cache.v_scales if q4 else cache.v)[p, 1, 100 % page, 0] = math.nan
    out, lse = af.paged_decode(randn(2, 8, d, seed=27), cache, i32(lens))
    bad = torch.isnan(out).any(-1)
    assert bad[1, 4:].all() and not bad[0].any() and not bad[1, :4].any()
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("q4", [False, True])
def test_decode_strides_outputs_and_workspace(q4):
    """q and out as views, pools as views, a shared page, own workspace, no LSE."""
    Hq, Hkv, page, d, lens = 8, 2, 32, 128, [100, 75, 64]
    base = make_cache(lens, 2 * Hkv, page, d, q4, seed=28, garbage=False)
    half = lambda x: None if x is None else x[:, 1::2]  # noqa: E731
    table = base.page_table.clone()
    table[1, 0] = table[0, 0]  # a common prefix
    wide = torch.full((3, 9), -1, dtype=torch.int32, device=DEV)
    wide[:, 2:2 + table.shape[1]] = table
    cache = af.PagedCache(half(base.k), half(base.v), wide[:, 2:2 + table.shape[1]], half(base.k_scales), half(base.v_scales))
    qbig = randn(3, 2, Hq, d + 8, seed=29)
    q = qbig[:, 1, :, 8:]
    obig = torch.full((Hq, 3, 2, d), 5.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(af.paged_decode_workspace_size(Hq, Hkv, d, cache.format) + 64, dtype=torch.uint8, device=DEV)
    out, lse = af.paged_decode(q, cache, i32(lens), out=obig[:, :, 0].transpose(0, 1), with_lse=False, workspace=ws)
    assert lse is None and out.data_ptr() == obig.data_ptr()
    lse2 = torch.empty(3, Hq, device=DEV)
    out2, _ = af.paged_decode(q, cache, i32(lens), lse=lse2)
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and (obig[:, :, 1] == 5).all()
    P.check_decode((out2, lse2), P.decode(q, cache, i32(lens), d ** -0.5, 1e4))


@pytest.mark.parametrize("q4", [False, True])
def test_offsets_past_32_bits(q4):
    """Pages whose byte offset passes 2^32, written and read."""
    Hq, Hkv, page, d, N = 8, 8, 128, 128, 300
    per = Hkv * page * (d // 2 if q4 else 2 * d)
    n = (1 << 32) // per + 40
    if torch.cuda.mem_get_info()[0] < 6 * n * per:
        pytest.skip("not enough device memory")
    table = i32([[n - 1, n - 9, 0], [n - 2, 1, n - 30]])
    cache = af.PagedCache.empty(n, Hkv, page, d, table, q4=q4)
    k, v = randn(2, Hkv, N, d, seed=30), randn(2, Hkv, N, d, seed=31)
    af.paged_append(cache, k, v, i32([3, 0]), rope_theta=5e5)
    # the same rows in a small cache
    small = af.PagedCache.empty(6, Hkv, page, d, i32([[0, 1, 2], [3, 4, 5]]), q4=q4)
    af.paged_append(small, k, v, i32([3, 0]), rope_theta=5e5)
    for c in (cache, small):
        af.paged_append(c, k[:, :, :3], v[:, :, :3], i32([0, 300]), rope_theta=5e5)
    q = randn(2, Hq, d, seed=32)
    lens = i32([303, 303])
    a, b = (af.paged_decode(q, c, lens, rope_theta=5e5) for c in (cache, small))
    ga, gb = (af.paged_gather(c, None, lens, 303) for c in (cache, small))
    torch.cuda.synchronize()
    assert af.device_status() == 0
    for x, y in zip(a + ga, b + gb):
        assert torch.equal(x, y)


# ---------------------------------------------------------------------------------------------
# values on the device that are out of range; streams, graphs, repeated calls
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("q4", [False, True])
def test_bad_pages_and_lengths_are_skipped_and_reported(q4):
    Hkv, page, d, lens = 2, 16, 64, [100, 100, 40]
    cache = make_cache(lens, Hkv, page, d, q4, seed=33, garbage=False)
    q = randn(3, 4, d, seed=34)
    good = af.paged_decode(q, cache, i32(lens))
    gathered = af.paged_gather(cache, None, i32([100, 100, 40]), 100)
    assert af.device_status() == 0
    for bad in (-1, cache.num_pages, 1 << 30):
        table = cache.page_table.clone()
        table[1, 2] = bad
        c = af.PagedCache(cache.k, cache.v, table, cache.k_scales, cache.v_scales)
        out, lse = af.paged_decode(q, c, i32(lens))
        assert af.device_status() == PAGE_RANGE and af.device_status() == 0
        assert torch.equal(out[[0, 2]], good[0][[0, 2]]) and torch.isfinite(out).all() and torch.isfinite(lse).all()
        before = [x.clone() for x in (c.k, c.v)]
        k, v = af.paged_gather(c, None, i32(lens), 100)
        assert af.device_status() == PAGE_RANGE
        assert (k[1, :, 32:48] == 0).all() and torch.equal(k[1, :, 48:], gathered[0][1, :, 48:])
        x = randn(3, Hkv, 8, d, seed=35)
        af.paged_append(c, x, x, i32([0, 36, 0]), i32([0, 8, 0]))
        assert af.device_status() == PAGE_RANGE
        assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1])
    # lengths and counts outside their ranges: clamped
    cap = cache.max_pages * page
    out, lse = af.paged_decode(q, cache, i32([-3, 100, 40]))
    assert af.device_status() == PAGE_RANGE
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all() and torch.equal(out[1:], good[0][1:])
    af.paged_decode(q, cache, i32([cap + 1, 100, 2**31 - 1]))
    assert af.device_status() == PAGE_RANGE
    before = cache.k.clone()
    x = randn(3, Hkv, 2, d, seed=36)
    af.paged_append(cache, x, x, i32([-1, cap, 2**31 - 1]), i32([2, 1, 2]), rope_mode=af.ROPE_NONE)
    assert af.device_status() == PAGE_RANGE
    p0 = cache.page_table[0, 0].item()  # sequence 0's second row is position 0 and in range
    before[p0, :, 0] = cache.k[p0, :, 0]
    assert torch.equal(cache.k, before)
    af.paged_append(cache, x, x, i32([0, 0, 0]), i32([3, -1, 0]))
    assert af.device_status() == PAGE_RANGE


@pytest.mark.parametrize("q4", [False, True])
def test_captured_steps_follow_the_device_lengths(q4):
    """One captured step (append, decode), replayed while lengths and tokens change on the
    device; a second graph shares the workspace; eager calls on a side stream agree."""
    B, Hq, Hkv, page, d, steps = 3, 8, 2, 16, 128, 40
    first = [0, 14, 170]
    cache = make_cache([n + steps for n in first], Hkv, page, d, q4, seed=37, garbage=False)
    ks, vs, qs = (randn(steps, B, h, d, seed=38 + i) for i, h in enumerate((Hkv, Hkv, Hq)))
    ws = torch.empty(max(16, af.paged_decode_workspace_size(Hq, Hkv, d, cache.format)), dtype=torch.uint8, device=DEV)
    k, v, q = ks[0].clone(), vs[0].clone(), qs[0].clone()
    lens = i32(first)

    def step():
        start = lens.clone()
        lens.add_(1)
        af.paged_append(cache, k[:, :, None], v[:, :, None], start, rope_theta=5e5)
        return af.paged_decode(q, cache, lens, rope_theta=5e5, workspace=ws)

    step()  # library set-up happens before a capture
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        graphs.append((g, got))
    lens.copy_(i32(first))
    outs = []
    for n in range(steps):
        for x, y in ((k, ks), (v, vs), (q, qs)):
            x.copy_(y[n])
        g, got = graphs[n % 2]
        g.replay()
        outs.append([x.clone() for x in got])
    torch.cuda.synchronize()
    assert af.device_status() == 0
    assert lens.tolist() == [n + steps for n in first]
    # the same steps, eagerly, on another stream
    lens.copy_(i32(first))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for n in range(steps):
            for x, y in ((k, ks), (v, vs), (q, qs)):
                x.copy_(y[n])
            out, lse = step()
            assert torch.equal(out, outs[n][0]) and torch.equal(lse, outs[n][1])
    side.synchronize()


@pytest.mark.parametrize("q4", [False, True])
def test_decode_results_do_not_vary(q4):
    cache = make_cache([5000, 17, 900], 2, 64, 128, q4, seed=41)
    q = randn(3, 16, 128, seed=42)
    first = af.paged_decode(q, cache, i32([5000, 17, 900]))
    for _ in range(20):
        again = af.paged_decode(q, cache, i32([5000, 17, 900]))
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("q4", [False, True])
def test_prompt_then_decode_together(q4):
    """A run as a server makes it: a padded batch of prompts through the forward and into the
    cache, then tokens one at a time; each step equals the dense forward over the values that
    the cache holds, with the rotation already in them."""
    B, Hq, Hkv, d, page, N, steps, theta = 3, 8, 2, 128, 48, 150, 5, 5e5
    plen = [150, 1, 77]
    table, n = table_for([x + steps for x in plen], page, 43)
    cache = af.PagedCache.empty(n, Hkv, page, d, table, q4=q4)
    for x in (cache.k, cache.v) + ((cache.k_scales, cache.v_scales) if q4 else ()):
        x.view(torch.uint8).fill_(0xFF)  # NaN, as uninitialised memory may be
    q, k, v = randn(B, Hq, N + steps, d, seed=44), randn(B, Hkv, N + steps, d, seed=45), randn(B, Hkv, N + steps, d, seed=46)
    prompt, _ = af.fwd(q[:, :, :N].contiguous(), k[:, :, :N].contiguous(), v[:, :, :N].contiguous(), rope_theta=theta,
                       variant=af.Variant(mask=af.MASK_CAUSAL))
    af.paged_append(cache, k[:, :, :N], v[:, :, :N], i32([0] * B), i32(plen), rope_theta=theta)
    lens = list(plen)
    for t in range(steps):
        row = lambda x: torch.stack([x[b, :, lens[b]] for b in range(B)])  # noqa: E731
        af.paged_append(cache, row(k)[:, :, None], row(v)[:, :, None], i32(lens), rope_theta=theta)
        lens = [x + 1 for x in lens]
        qt = torch.stack([q[b, :, lens[b] - 1] for b in range(B)])
        out, lse = af.paged_decode(qt, cache, i32(lens), rope_theta=theta)
        P.check_decode((out, lse), P.decode(qt, cache, i32(lens), d ** -0.5, theta))
        kd, vd = af.paged_gather(cache, None, i32(lens), max(lens))
        for b in range(B):
            L = lens[b]
            o, l = af.decode(qt[b:b + 1], kd[b:b + 1, :, :L].contiguous(), vd[b:b + 1, :, :L].contiguous(), L - 1, rope_theta=theta)
            # the dense decode rounds the rotated q, and here the 4-bit values, to bf16: both
            # within its documented bar
            assert (o[0].float() - out[b].float()).abs().max().item() <= 2e-2
            assert (l[0] - lse[b]).abs().max().item() <= 2e-2
            if not q4:  # the token's row of the fused forward over the same sequence
                full, _ = af.fwd(*(x[b:b + 1, :, :L].contiguous() for x in (q, k, v)), rope_theta=theta,
                                 variant=af.Variant(mask=af.MASK_CAUSAL))
                assert (full[0, :, L - 1].float() - out[b].float()).abs().max().item() <= 2e-2
    assert torch.isfinite(prompt).all() and af.device_status() == 0


@pytest.mark.parametrize("q4", [False, True])
def test_calls_on_a_given_stream_own_what_they_allocate(q4):
    """A call on a busy stream is still queued when the caller goes on: memory that the call
    allocated may not reach the current stream's next tensors before it has run."""
    lens = [9000, 300]
    cache = make_cache(lens, 2, 64, 128, q4, seed=51)
    q, ln = randn(2, 8, 128, seed=52), i32(lens)
    want, rows = af.paged_decode(q, cache, ln), af.paged_gather(cache, None, ln, 9000)
    n = af.paged_decode_workspace_size(8, 2, 128, cache.format)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = af.paged_decode(q, cache, ln, stream=side)
        dense = af.paged_gather(cache, None, ln, 9000, stream=side)
        keep = [torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(4)]
        side.synchronize()
        torch.cuda.synchronize()
        for x, y in zip(got + dense, want + rows):
            assert torch.equal(x, y)
        assert all((x == 0x7F).all() for x in keep)
        del keep


@pytest.mark.parametrize("q4", [False, True])
def test_steps_on_two_streams_at_once(q4):
    """Two batches over one pool of pages, each stepped on a stream of its own."""
    Hkv, Hq, page, d, steps = 2, 16, 32, 128, 12
    first = [[700, 0, 33, 5000], [1, 2900, 64, 128]]
    both = make_cache([n + steps for part in first for n in part], Hkv, page, d, q4, seed=53, garbage=False)
    copies = [x.clone() for x in both._tensors if x is not None]
    ks, vs, qs = (randn(2, steps, 4, h, d, seed=54 + i) for i, h in enumerate((Hkv, Hkv, Hq)))

    def run(streams):
        outs = [[], []]
        caches = [af.PagedCache(both.k, both.v, both.page_table[4 * i:4 * i + 4], both.k_scales, both.v_scales) for i in (0, 1)]
        lens = [i32(x) for x in first]
        torch.cuda.synchronize()
        for n in range(steps):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    start = lens[i].clone()
                    lens[i].add_(1)
                    af.paged_append(caches[i], ks[i, n][:, :, None], vs[i, n][:, :, None], start, rope_theta=5e5)
                    outs[i].append(af.paged_decode(qs[i, n], caches[i], lens[i], rope_theta=5e5))
        torch.cuda.synchronize()
        return outs

    one = torch.cuda.current_stream()
    alone = run([one, one])
    for x, y in zip((x for x in both._tensors if x is not None), copies):
        x.copy_(y)
    at_once = run([torch.cuda.Stream(), torch.cuda.Stream()])
    for a, b in zip(alone, at_once):
        for x, y in zip(a, b):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    assert af.device_status() == 0


@pytest.mark.parametrize("q4", [False, True])
def test_decode_many_sequences_of_large_groups(q4):
    """More items than CTAs with two passes of query heads each, the second of them ragged."""
    r = random.Random(55)
    lens = [r.choice([0, 1, r.randint(1, 64), r.randint(1, 700)]) for _ in range(90)]
    run_decode(lens, 80, 4, 32, 64, q4, theta=1e4, seed=55)
    run_decode(lens[:40] + [4000], 40, 2, 16, 128, q4, seed=56)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("pages", [10, 20, 40, 41, 64])
def test_decode_caches_of_short_sequences(q4, pages):
    """Capacities on both sides of where sequences are cut, for few and for many of them."""
    page, Hkv, Hq, d = 16, 2, 6, 128
    full = pages * page
    lens = [full, 0, 1, full - 1, 17, full // 2] + [37] * 60
    wide = make_cache(lens, Hkv, page, d, q4, seed=61 + pages)
    slopes = torch.tensor([0.5, 0.25, 0.0, 2.0 ** -6, 2.0 ** -9, -0.125], device=DEV)
    for n in (1, 6, len(lens)):
        small = af.PagedCache(wide.k, wide.v, wide.page_table[:n, :pages], wide.k_scales, wide.v_scales)
        for kw in (dict(theta=1e4), dict(window=100, slopes=slopes)):
            run_decode(lens[:n], Hq, Hkv, page, d, q4, cache=small, seed=62, **kw)


@pytest.mark.parametrize("q4", [False, True])
def test_sequences_may_share_pages(q4):
    """One row of the table for all sequences: its stride is 0."""
    own = make_cache([600], 2, 16, 128, q4, seed=57)
    shared = af.PagedCache(own.k, own.v, own.page_table.expand(3, -1), own.k_scales, own.v_scales)
    lens = [600, 37, 599]
    got = run_decode(lens, 4, 2, 16, 128, q4, theta=1e4, cache=shared, seed=8)
    rows = af.PagedCache(own.k, own.v, shared.page_table.clone(), own.k_scales, own.v_scales)
    again = run_decode(lens, 4, 2, 16, 128, q4, theta=1e4, cache=rows, seed=8)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    first, count = [0, 16, 500], [100, 21, 99]
    for dense, which in zip(af.paged_gather(shared, i32(first), i32(count), 100), "kv"):
        pool = P.values(shared, which)
        for b in range(3):
            assert torch.equal(dense[b, :, :count[b]], P.rows(pool, shared.page_table, b, first[b], count[b]).float().bfloat16())
            assert (dense[b, :, count[b]:] == 0).all()


@pytest.mark.parametrize("q4", [False, True])
def test_windows_past_the_sequence_are_none(q4):
    lens = [700, 1, 130]
    cache = make_cache(lens, 2, 32, 64, q4, seed=59)
    q = randn(3, 4, 64, seed=60)
    want = af.paged_decode(q, cache, i32(lens))
    for window in (700, 1 << 24, (1 << 31) - 1, 1 << 31, 1 << 40):
        got = af.paged_decode(q, cache, i32(lens), window=window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), window


def test_refusals_on_the_gpu():
    """What only a CUDA tensor lets the binding see; every call fails before a launch."""
    Hkv, page, d = 2, 16, 64
    table = i32([[0, 1], [2, 3]])
    c = af.PagedCache.empty(4, Hkv, page, d, table)
    c4 = af.PagedCache.empty(4, Hkv, page, d, table, q4=True)
    k = randn(2, Hkv, 3, d, seed=0)
    q = randn(2, 4, d, seed=0)
    ok = i32([0, 0])
    with pytest.raises(TypeError, match="expected a PagedCache"):
        af.paged_append((c.k, c.v), k, k, ok)
    with pytest.raises(ValueError, match="belong to the 4-bit format"):
        af.PagedCache(c.k, c.v, table, c4.k_scales, c4.v_scales)
    with pytest.raises(TypeError, match="cache k_scales"):
        af.PagedCache(c4.k, c4.v, table)
    with pytest.raises(TypeError, match="page_table: dtype"):
        af.PagedCache(c.k, c.v, table.long())
    with pytest.raises(ValueError, match="rows must be contiguous"):
        af.PagedCache(c.k, c.v, table.t())
    with pytest.raises(ValueError, match="cache v: shape"):
        af.PagedCache(c.k, c.v[1:], table)
    with pytest.raises(ValueError, match="k: shape"):
        af.paged_append(c, k[:1], k[:1], ok)
    with pytest.raises(ValueError, match="v: shape"):
        af.paged_append(c, k, k[:, :, :2], ok)
    with pytest.raises(TypeError, match="start"):
        af.paged_append(c, k, k, None)
    with pytest.raises(TypeError, match="start: dtype"):
        af.paged_append(c, k, k, ok.long())
    with pytest.raises(ValueError, match="count: shape"):
        af.paged_append(c, k, k, ok, ok[:1])
    with pytest.raises(ValueError, match="start: on cpu"):
        af.paged_append(c, k, k, ok.cpu())
    with pytest.raises(TypeError, match="lens"):
        af.paged_decode(q, c, None)
    with pytest.raises(ValueError, match="q: shape"):
        af.paged_decode(q[..., :32], c, ok)
    with pytest.raises(ValueError, match="alibi_slopes: shape"):
        af.paged_decode(q, c, ok, alibi_slopes=torch.ones(3, device=DEV))
    for bad in (dict(scale=0.0), dict(scale=math.inf), dict(window=-1), dict(rope_theta=0.0)):
        with pytest.raises(af.AttnfuseError) as e:
            af.paged_decode(q, c, ok, **bad)
        assert e.value.code == 1
    for call in (lambda: af.paged_decode(q, c, ok, rope_mode=af.ROPE_PREROTATE),
                 lambda: af.paged_append(c, k, k, ok, rope_mode=9),
                 lambda: af.paged_decode(randn(2, 3, d, seed=1), c, ok),
                 lambda: af.paged_append(af.PagedCache(c.k[:, :, :8], c.v[:, :, :8], table), k, k, ok)):
        with pytest.raises(af.AttnfuseError) as e:
            call()
        assert e.value.code == 2
    for call in (lambda: af.paged_append(c, k[..., ::2].expand(2, Hkv, 3, 32)[..., :0], k, ok),
                 lambda: af.paged_gather(c, ok, ok, 0),
                 lambda: af.paged_decode(torch.empty(2 * 4 * d + 1, dtype=torch.bfloat16, device=DEV)[1:].view(2, 4, d), c, ok),
                 lambda: af.paged_append(af.PagedCache(c4.k.transpose(1, 2).contiguous().transpose(1, 2), c4.v, table,
                                                       c4.k_scales, c4.v_scales), k, k, ok),
                 lambda: af.paged_append(c, k[:, :, :1].expand(2, Hkv, 3, d), k, ok)):
        with pytest.raises((af.AttnfuseError, ValueError)):
            call()
    assert af.device_status() == 0
