"""GPU parity: rotary positions on several axes against a 64-bit statement, their inverse, and their
place in front of the forward, the backward and the paged caches."""
import math

import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af
from attention_attn_fwd_bwd_gb300 import combinators as C

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
DEV = torch.device("cuda")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    af.load()


def randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator(DEV).manual_seed(seed), device=DEV).bfloat16()


def positions(axes, B, N, lo, hi, seed):
    return torch.randint(lo, hi, (axes, B, N), generator=torch.Generator(DEV).manual_seed(seed), device=DEV, dtype=torch.int32)


def frequencies(sections, theta, interleaved, own):
    """(axis, frequency) of each pair."""
    left = [list(range(n)) for n in sections]
    order = []
    if interleaved:
        while any(left):
            order += [(a, q.pop(0)) for a, q in enumerate(left) if q]
    else:
        order = [(a, j) for a, q in enumerate(left) for j in q]
    h = len(order)
    return [(a, theta ** -(j / sections[a] if own else i / h)) for i, (a, j) in enumerate(order)]


def angles(pos, sections, theta=1e4, interleaved=False, own=False):
    """[B, 1, N, d/2] in 64 bits."""
    fr = frequencies(sections, theta, interleaved, own)
    f = torch.tensor([x for _, x in fr], dtype=torch.float64, device=DEV)
    p = pos[[a for a, _ in fr]].permute(1, 2, 0).double()
    return (p * f)[:, None]


def turned(x, ang):
    x = x.double()
    h = x.shape[-1] // 2
    c, s = torch.cos(ang), torch.sin(ang)
    return torch.cat((x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s), -1)


def check(got, x, ang, angle_error=0.0):
    """Half a step of bf16, 2^-9 of the value (2^-8 of its binade's floor), the two roundings to fp32
    and bf16 (2^-24 more) and what the reference's own angles are off by."""
    want = turned(x, ang)
    h = x.shape[-1] // 2
    size = x.double().abs()
    size = (size[..., :h] + size[..., h:]).repeat(*(1,) * (x.dim() - 1), 2)
    tol = (2.0 ** -8 + 2.0 ** -23) * want.abs() + (2.0 ** -30 + angle_error) * size + 2.0 ** -133
    over = (got.double() - want).abs() - tol
    assert over.max().item() <= 0, over.max().item()


CASES = [  # d, sections, interleaved, own spectrum, B, Hq, Hk, N
    (128, (16, 24, 24), False, False, 2, 32, 8, 37),
    (128, (24, 20, 20), True, False, 1, 8, 1, 301),
    (64, (16, 16), True, True, 3, 16, 16, 129),
    (64, (8, 10, 13, 1), True, True, 2, 3, 1, 65),
    (64, (1, 31), False, True, 5, 4, 4, 1),
    (128, (64,), False, False, 1, 1, 0, 1),
    (128, (5, 7, 50, 2), False, False, 64, 32, 8, 1),
    (64, (32,), True, False, 1, 40, 8, 2049),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("d, sections, interleaved, own, B, Hq, Hk, N", CASES)
def test_against_64_bits(d, sections, interleaved, own, B, Hq, Hk, N, inverse):
    q = randn(B, Hq, N, d, seed=1)
    k = randn(B, Hk, N, d, seed=2) if Hk else None
    pos = positions(len(sections), B, N, -40, 5000, 3)
    gq, gk = af.rope_axes(q, k, pos, sections, rope_theta=5e5, interleaved=interleaved, own_spectrum=own, inverse=inverse)
    ang = angles(pos, sections, 5e5, interleaved, own) * (-1 if inverse else 1)
    check(gq, q, ang, 5000 * 2.0 ** -51)
    if Hk:
        check(gk, k, ang, 5000 * 2.0 ** -51)
    else:
        assert gk is None


@pytest.mark.parametrize("theta", [0.05, 1.0, 1e4, 5e6])
def test_any_position_of_32_bits(theta):
    far = [0, 1, -1, 4095, 4096, -4096, 1 << 24, (1 << 24) + 1, -(1 << 24), -(1 << 24) - 1, 123456789, -987654321,
           (1 << 31) - 1, -(1 << 31)]
    N = len(far)
    pos = torch.tensor([far, far[::-1]], dtype=torch.int32, device=DEV)[:, None]
    x = randn(1, 2, N, 64, seed=5)
    got, _ = af.rope_axes(x, None, pos, (16, 16), rope_theta=theta)
    # in fractions, since 53 bits of a frequency alone would leave an angle of 2^31 f by 2^-22 off
    from fractions import Fraction

    pi = Fraction(884279719003555, 1 << 48) + Fraction(4967757600021511, 1 << 105)
    root = Fraction(float(torch.tensor(theta, dtype=torch.float32)))
    for _ in range(5):  # theta^(1/32), to 2^-190
        root = Fraction(math.isqrt(int(root * (1 << 400))), 1 << 200)
    ang = torch.empty(1, 1, N, 32, dtype=torch.float64)
    for i in range(32):
        turn = 1 / root ** i / (2 * pi)
        for n in range(N):
            t = pos[i // 16, 0, n].item() * turn
            ang[0, 0, n, i] = float(2 * pi * (t - math.floor(t)))
    check(got, x, ang.to(DEV), 2.0 ** -48)


def test_strides_broadcast_positions_and_in_place():
    B, N, Hq, Hk, d = 2, 77, 12, 4, 128
    qkv = randn(B, N, Hq + 2 * Hk, d, seed=6).transpose(1, 2)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    pos = positions(3, 1, N, 0, 900, 7)[:, 0]
    ang = angles(pos[:, None].expand(3, B, N), (16, 24, 24))
    gq, gk = af.rope_axes(q, k, pos, (16, 24, 24))
    assert gq.is_contiguous() and gk.is_contiguous()
    check(gq, q, ang), check(gk, k, ang)
    wide = positions(3, B, 2 * N, 0, 900, 8)
    eq, _ = af.rope_axes(q, None, wide[:, :, ::2], (16, 24, 24))
    check(eq, q, angles(wide[:, :, ::2], (16, 24, 24)))
    v = qkv[:, Hq + Hk:].clone()
    rq, rk = af.rope_axes(q, k, pos, (16, 24, 24), q_out=q, k_out=k)
    assert rq is q and rk is k and torch.equal(q, gq) and torch.equal(k, gk) and torch.equal(qkv[:, Hq + Hk:], v)


def test_infinities_and_nan_stay_in_their_pairs():
    x = randn(1, 1, 4, 64, seed=9)
    x[0, 0, 1, 3], x[0, 0, 2, 40] = math.inf, math.nan
    pos = positions(1, 1, 4, 1, 50, 10)
    got, _ = af.rope_axes(x, None, pos, (32,))
    bad = ~torch.isfinite(got[0, 0])
    want = torch.zeros_like(bad)
    want[1, 3] = want[1, 35] = want[2, 8] = want[2, 40] = True
    assert torch.equal(bad, want)


def test_keys_are_those_that_an_append_stores():
    B, H, N, d = 2, 3, 50, 128
    k, v = randn(B, H, N, d, seed=11), randn(B, H, N, d, seed=12)
    start = torch.tensor([5, 1000], dtype=torch.int32, device=DEV)
    table = torch.arange(2 * 70, dtype=torch.int32, device=DEV).view(2, 70)
    a, b = (af.PagedCache.empty(140, H, 16, d, table) for _ in "ab")
    for c in (a, b):
        c.k.zero_(), c.v.zero_()
    af.paged_append(a, k, v, start, rope_theta=5e5)
    _, rk = af.rope_axes(k, k, (start[:, None] + torch.arange(N, device=DEV, dtype=torch.int32))[None], (64,), rope_theta=5e5)
    af.paged_append(b, rk, v, start, rope_mode=af.ROPE_NONE)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


def test_captured_and_replayed_with_other_positions_on_another_stream():
    q, k = randn(2, 4, 33, 64, seed=13), randn(2, 2, 33, 64, seed=14)
    pos = positions(2, 2, 33, 0, 100, 15)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        af.rope_axes(q, k, pos, (16, 16), q_out=qo, k_out=ko)
    pos.copy_(positions(2, 2, 33, 0, 100, 16))
    g.replay()
    torch.cuda.synchronize()
    check(qo, q, angles(pos, (16, 16))), check(ko, k, angles(pos, (16, 16)))
    with torch.cuda.stream(side):
        q2 = randn(2, 4, 33, 64, seed=17)
    gq, _ = af.rope_axes(q2, None, pos, (16, 16), stream=side)
    side.synchronize()
    check(gq, q2, angles(pos, (16, 16)))


def test_refusals():
    q, pos = randn(1, 4, 8, 64, seed=1), positions(2, 1, 8, 0, 9, 1)
    for bad in (dict(sections=(16, 15)), dict(sections=(0, 32)), dict(sections=(32,)), dict(positions=pos.long()),
                dict(positions=pos.cpu()), dict(positions=pos[:, :, :7]), dict(k=randn(1, 4, 7, 64, seed=2)),
                dict(k=q[:, :0]), dict(k_out=q), dict(q_out=q[:, :2]), dict(rope_theta=-1.0), dict(q=q.float())):
        args = dict(q=q, k=None, positions=pos, sections=(16, 16)) | bad
        with pytest.raises((ValueError, TypeError, af.AttnfuseError)):
            af.rope_axes(**args)


# ---------------------------------------------------------------------------------------------
# in front of the attention, and its gradients
# ---------------------------------------------------------------------------------------------
def _attend64(q, k, v, ang, causal):
    q, k, v = turned(q, ang), turned(k, ang), v.double()
    g = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    x = q @ k.transpose(-1, -2) / math.sqrt(q.shape[-1])
    if causal:
        N = x.shape[-1]
        x = x.masked_fill(torch.ones(N, N, device=x.device).triu(1).bool(), -math.inf)
    return torch.softmax(x, -1) @ v


@pytest.mark.parametrize("d, sections, interleaved, own", [(64, (16, 16), True, True), (128, (16, 24, 24), False, False)])
def test_training_step_through_the_combinator(d, sections, interleaved, own):
    B, Hq, Hk, N = 2, 4, 2, 200
    q, k, v = (randn(B, h, N, d, seed=20 + i).requires_grad_() for i, h in enumerate((Hq, Hk, Hk)))
    pos = positions(len(sections), B, N, 0, 300, 23)
    attn = C.attention(C.rope_axes(pos, sections, theta=1e4, interleaved=interleaved, own_spectrum=own), C.causal())
    out = attn(q, k, v)
    dout = randn(B, Hq, N, d, seed=24)
    grads = torch.autograd.grad(out, (q, k, v), dout)
    ref = [x.detach().double().requires_grad_() for x in (q, k, v)]
    want = _attend64(*ref, angles(pos, sections, 1e4, interleaved, own), True)
    ref_grads = torch.autograd.grad(want, ref, dout.double())
    # roundings to bf16 along the way (rotated rows, weights, dS, gradients, their turn back): each
    # 2^-9 of its value at most, ten of them; by norm
    for got, ref_ in zip((out, *grads), (want, *ref_grads)):
        assert (got.double() - ref_).norm() <= 10 * 2.0 ** -9 * ref_.norm()


def test_gradient_is_the_inverse_rotation_and_matches_differences():
    B, H, N, d = 1, 2, 9, 64
    x = randn(B, H, N, d, seed=30)
    dy = randn(B, H, N, d, seed=31)
    pos = positions(3, B, N, 0, 500, 32)
    args = (pos, (8, 12, 12))
    dx, _ = af.rope_axes(dy, None, *args, inverse=True)
    # the map is linear: <R e, dy> = <e, R^T dy> for the differences e = 2^k in one place at a time
    for i in (0, 7, 31, 32, 63):
        e = torch.zeros_like(x)
        e[..., i] = 2.0 ** 4
        up, _ = af.rope_axes(x * 0 + e, None, *args)
        slope = (up.double() * dy.double()).sum(-1) / 2.0 ** 4
        size = dy.double().abs().sum(-1)
        assert ((slope - dx[..., i].double()).abs() <= 2.0 ** -8 * 2 * size).all()


def test_positions_changed_before_the_backward_are_noticed():
    q, k, v = (randn(1, 2, 64, 64, seed=40 + i).requires_grad_() for i in range(3))
    pos = positions(2, 1, 64, 0, 50, 43)
    out = C.attention(C.rope_axes(pos, (16, 16)), C.causal())(q, k, v)
    pos.add_(1)
    with pytest.raises(RuntimeError):
        out.sum().backward()
