"""GPU parity of the paged decode where weights and values are of very uneven size: keys that carry
all of the weight, or none of it, beside values far larger or smaller than the others."""
import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af
from tests import _paged as P

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
DEV = torch.device("cuda")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    af.load()
    assert af.device_status() == 0


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator(DEV).manual_seed(seed), device=DEV)


def filled(k, v, page, q4):
    """A cache of one page run per sequence that holds rows k, v [B, Hkv, L, d] as they are."""
    B, Hkv, L, d = k.shape
    pages = -(-L // page)
    table = torch.randperm(B * pages, generator=torch.Generator().manual_seed(L)).int().view(B, pages).to(DEV)
    cache = af.PagedCache.empty(B * pages, Hkv, page, d, table, q4=q4)
    af.paged_append(cache, k.bfloat16(), v.bfloat16(), i32([0] * B), rope_mode=af.ROPE_NONE)
    return cache


def group_floor(q, cache, lens, scale, window):
    """What weights below fp16's normal range may add to an element's tolerance, [B, Hq, d].

    A weight w = p * step of a 4-bit cache is one fp16 of w * mul, mul a power of two that takes the
    largest w so far of its head and group to 2^4 or more. Below 2^-14 it is off by at most 2^-25:
    in w, by 2^-25 / mul <= 2^-29 max w. A code is at most 7, and the key of a group's largest value
    has one of 7, so n keys add at most n 2^-29 max(7 w) = n 2^-29 max over the keys and the group's
    elements of p|v|. An element's own sum of p|v| may be less than that, where its code is 0 in the
    key that carries the weight."""
    B, Hq, d = q.shape
    k64, v64 = P.values(cache, "k"), P.values(cache, "v")
    floor = torch.zeros(B, Hq, d, dtype=torch.float64, device=q.device)
    for b, L in enumerate(lens.tolist()):
        first = max(0, L - window) if window else 0
        k, v = (P.rows(x, cache.page_table, b, first, L - first) for x in (k64, v64))
        p = torch.softmax(scale * torch.einsum("hgc,hnc->hgn", q[b].double().view(cache.Hkv, -1, d), k), -1)
        size = v.abs().unflatten(-1, (-1, P.GROUP)).amax(-1)  # [Hkv, n, groups]
        most = torch.stack([(p[..., None] * size[:, None])[:, i].amax(1) for i in range(p.shape[1])], 1)
        floor[b] = ((L - first) * 2.0 ** -29 * most).repeat_interleave(P.GROUP, -1).view(Hq, d)
    return floor


def check(q, cache, lens, scale, window=0):
    got = af.paged_decode(q, cache, lens, scale=scale, rope_mode=af.ROPE_NONE, window=window)
    torch.cuda.synchronize()
    assert af.device_status() == 0
    o, l, to, tl = P.decode(q, cache, lens, scale, None, window)
    if cache.q4:
        to = to + group_floor(q, cache, lens, scale, window)
    P.check_decode(got, (o, l, to, tl))


def steered(B, Hq, Hkv, L, d, seed, spread):
    """q, k, v with scores under control: element 0 of every query is 8 and of every key 0, and the
    other elements are normal (times `spread` in the keys), so that a key whose element 0 is x
    scores 8 x scale more than its others make it."""
    q, k, v = randn(B, Hq, d, seed=seed), spread * randn(B, Hkv, L, d, seed=seed + 1), randn(B, Hkv, L, d, seed=seed + 2)
    q[..., 0] = 8
    k[..., 0] = 0
    return q.bfloat16(), k, v


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("Hq,d", [(8, 128), (3, 128), (12, 128), (8, 64)])
@pytest.mark.parametrize("log2_size", [6, 12, 16, 20, 24, 40])
def test_large_values_of_keys_without_weight(q4, Hq, d, log2_size):
    """One key's values are 2^6 to 2^40 times the others' and its score is about 60 below theirs,
    so that it adds nothing: what the other keys add keeps its bits, wherever the key stands."""
    scale = d ** -0.5
    for L in (20, 500, 5000):
        where = [0, L // 2, L - 1]
        q, k, v = steered(3, Hq, 1, L, d, 70 + L, 1.0)
        for b, n in enumerate(where):
            k[b, :, n] = 0
            k[b, :, n, 0] = -60 / (8 * scale)
            v[b, :, n] *= 2.0 ** log2_size
        check(q, filled(k, v, 64, q4), i32([L] * 3), scale)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("Hq,d", [(8, 128), (2, 128), (16, 64)])
def test_large_values_that_some_heads_take(q4, Hq, d):
    """The same key has all of the weight of every second head of its group and none of the
    others'."""
    scale = d ** -0.5
    for L, log2_size in ((300, 18), (3000, 22)):
        q, k, v = steered(2, Hq, 1, L, d, 80 + L, 1.0)
        q[:, 1::2, 0] = -8
        for b, n in enumerate((3, L - 2)):
            k[b, :, n] = 0
            k[b, :, n, 0] = -60 / (8 * scale)
            v[b, :, n] *= 2.0 ** log2_size
        check(q, filled(k, v, 16, q4), i32([L] * 2), scale)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("Hq,d", [(8, 128), (4, 64)])
@pytest.mark.parametrize("log2_gap", [12, 18, 20, 24.6, 30, 40])
@pytest.mark.parametrize("sink", [2.0 ** -16, 1.0])
def test_dominating_key(q4, Hq, d, log2_gap, sink):
    """One key 2^12 to 2^40 above the others, which all score the same, with small values or ones
    like theirs (then what they add is below the output's own bits): their shares of the output
    are as small as each other. In 300 keys, which one CTA takes, and in 20000, which many do."""
    scale = d ** -0.5
    for L in (300, 20000):
        q, k, v = steered(3, Hq, 1, L, d, 90, 0.0)
        v = v.abs() + 0.5
        for b, n in enumerate((0, L // 2, L - 1)):
            k[b, :, n, 0] = log2_gap * 0.6931471805599453 / (8 * scale)
            v[b, :, n] *= sink
        check(q, filled(k, v, 16, q4), i32([L] * 3), scale)


@pytest.mark.parametrize("q4", [False, True])
def test_weights_that_fall_and_rise_along_a_sequence(q4):
    """Scores rise by 100 and fall again along the sequence while the values' sizes go the other
    way by 2^30: at every point the weight to come outgrows, or has outgrown, the one behind."""
    d, scale, L = 128, 128 ** -0.5, 4000
    n = torch.arange(L, device=DEV, dtype=torch.float32)
    up = 1 - (2 * n / (L - 1) - 1).abs()  # 0 .. 1 .. 0
    for sign in (1.0, -1.0):
        q, k, v = steered(2, 8, 2, L, d, 95, 0.3)
        k[..., 0] = sign * 100 / (8 * scale) * up
        v *= torch.exp2(-sign * 30 * up)[:, None]
        check(q, filled(k, v, 32, q4), i32([L, L // 3]), scale)
        check(q, filled(k, v, 32, q4), i32([L, L // 3]), scale, window=700)


@pytest.mark.parametrize("d", [64, 128])
def test_value_groups_of_zeros_beside_others(d):
    """Groups of values that are zero in all keys, or in all but one, of a 4-bit cache."""
    scale, L = d ** -0.5, 1500
    q, k, v = steered(2, 8, 1, L, d, 99, 1.0)
    v[..., :32] = 0
    v[1, :, 1200, :32] = 5
    v[0, :, 7, 5] = 2.0 ** -20
    check(q, filled(k, v, 16, True), i32([L, L - 13]), scale)
