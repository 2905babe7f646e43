"""GPU: the rotation of appended keys next to borders of its rounding. A key is R_p k rounded to
fp32 and then to bf16; keys are searched whose result would be another one if R_p k were off by
2^-31 (|x| + |y|), x and y the pair's elements, but not if it were off by the 2^-34 (|x| + |y|) that
the header allows."""
import decimal

import pytest
import torch

import attention_attn_fwd_bwd_gb300 as af

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
DEV = torch.device("cuda")
PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from attention_attn_fwd_bwd_gb300 import _build

    _build.build()
    af.load()
    assert af.device_status() == 0


def cos_sin(pos, i, d, theta):
    """Within 2^-51: the turn in 60 digits, its fraction in 64 bits."""
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        turn = pos * (decimal.Decimal(theta).ln() * -2 * i / d).exp() / (2 * PI)
        a = torch.tensor(float((turn - turn.to_integral_value()) * 2 * PI), dtype=torch.float64)
    return torch.cos(a).item(), torch.sin(a).item()


def near_borders(pos, i, d, theta):
    """Pairs (x, y, their results) for position pos and pair i whose result is as above."""
    c, s = cos_sin(pos, i, d, theta)
    m = torch.arange(128, 256, device=DEV, dtype=torch.float64)
    y = torch.cat([m * 2.0 ** e for e in (-1, 0, 1)] + [-m * 2.0 ** e for e in (-1, 0, 1)])
    x, y = m[:, None].expand(-1, len(y)), y.expand(len(m), -1)
    size = x.abs() + y.abs()
    lo, hi = x * c - y * s, y * c + x * s
    row = lambda v: v.float().bfloat16()  # noqa: E731
    moved = lambda r: sum((row(v + r * size) != row(v - r * size)).int() for v in (lo, hi))  # noqa: E731
    hit = (moved(2.0 ** -31) > 0) & (moved(2.0 ** -34) == 0)
    return [(x[hit][n].item(), y[hit][n].item(), row(lo[hit])[n].item(), row(hi[hit])[n].item())
            for n in range(int(hit.sum()))]


def check(positions, d, theta):
    H, page = 8, 16
    cases = 0
    for pos in positions:
        k = torch.zeros(1, H, 1, d)
        want = torch.zeros(H, d)
        for i in range(d // 2):
            for h, (x, y, lo, hi) in enumerate(near_borders(pos, i, d, theta)[:H]):
                k[0, h, 0, i], k[0, h, 0, i + d // 2], want[h, i], want[h, i + d // 2] = x, y, lo, hi
                cases += 1
        table = torch.full((1, pos // page + 1), -1, dtype=torch.int32, device=DEV)
        table[0, -1] = 0
        cache = af.PagedCache.empty(1, H, page, d, table)
        start = torch.tensor([pos], dtype=torch.int32, device=DEV)
        k = k.bfloat16().to(DEV)
        af.paged_append(cache, k, k, start, rope_theta=theta)
        got = cache.k[0, :, pos % page].float().cpu()
        assert torch.equal(got, want), f"position {pos}: {(got != want).sum().item()} elements differ"
    assert cases >= len(positions)
    assert af.device_status() == 0


@pytest.mark.parametrize("d,theta", [(128, 1e4), (64, 5e5), (128, 5e5)])
def test_keys_next_to_a_border(d, theta):
    check([1, 2, 77, 500, 1023, 2500, 4095, 30000], d, theta)


@pytest.mark.parametrize("d,theta", [(128, 1e4), (64, 5e5), (128, 0.5), (64, 2.0 ** -16)])
def test_keys_next_to_a_border_at_far_positions(d, theta):
    """Where a rounding of the frequency itself is multiplied by the position."""
    top = 1 << 24
    check([top - 1, top - 2, top - 12345, 15_000_001, 12_345_678, 3_000_003, 1_000_000, 131_071], d, theta)
