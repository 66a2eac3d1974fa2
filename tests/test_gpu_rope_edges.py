"""Rotary positions: the precision of the sines and cosines and of f32 rows."""
from decimal import Decimal, getcontext
import math

import pytest
import torch

import attend_ref as ref

pytestmark = pytest.mark.gpu

getcontext().prec = 80
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.fixture(scope="module")
def moe():
    import expert_routing_grouped_gb300 as m
    return m


def half_unit(v):
    """Half a unit in the last place of f32 at v."""
    return math.ldexp(1.0, math.frexp(v)[1] - 25) if v else 0.0


@pytest.mark.parametrize("mscale", [1.0, 1.25, 0.4])
@pytest.mark.parametrize("inverse", [False, True])
def test_sines_and_cosines(moe, inverse, mscale):
    """u = 1, v = 0 gives mscale (cos, sin) itself: rounded once, but for the series' own
    roundings (the part past the first term is at most 0.081, rounded four and a half
    times: 2^-25.4), at any position and frequency.  The fraction of a turn that a
    position makes is cut at 2^-64, and 1 / (2 pi) after 126 bits of its own (2^66 / (2 pi)
    is above 2^63 and held to 2^-64): pos (2 pi 2^-64 + |f| 2^-127) radians."""
    g = torch.Generator()
    g.manual_seed(41)
    pos = [0, 1, -1, 7, 1000, 65535, 10 ** 6, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, -12345678]
    pos += torch.randint(-2 ** 31, 2 ** 31 - 1, (20,), generator=g).tolist()
    freqs = [1e6 ** (-2.0 * i / 64) for i in range(32)] + [1.0, 3.3, 6.25, 1000.1, 123456.7, 1e12, 1e30, 0.0, 2.0 ** -70,
                                                           math.pi / 4, math.pi / 2, -0.3, -1e5]
    n = len(freqs)
    x = torch.zeros(len(pos), 1, 2 * n, device="cuda")
    x[..., :n] = 1
    out = torch.empty_like(x)
    m = float(torch.tensor(mscale))   # as f32 holds it
    moe.rope(x, torch.tensor(pos, dtype=torch.int32, device="cuda"), torch.tensor(freqs, dtype=torch.float64, device="cuda"),
             len(pos), 1, 2 * n, out, mscale=mscale, inverse=inverse, dtype=0)
    out = out.cpu()
    for a, p in enumerate(pos):
        for b, f in enumerate(freqs):
            turns = Decimal(p) * Decimal(f) / (2 * PI)
            ang = float((turns - turns.to_integral_value()) * 2 * PI) * (-1 if inverse else 1)
            cut = abs(p) * (2 * math.pi * 2.0 ** -64 + abs(f) * 2.0 ** -127)
            for got, v in ((out[a, 0, b], m * math.cos(ang)), (out[a, 0, n + b], m * math.sin(ang))):
                assert abs(float(got) - v) <= half_unit(v) + m * (2.0 ** -25.4 + cut), (p, f)


@pytest.mark.parametrize("interleaved", [False, True])
def test_f32_rows(moe, interleaved):
    """f32 rows lose no more than f32 arithmetic with rounded sines and cosines does."""
    g = torch.Generator(device="cuda")
    g.manual_seed(42)
    T, H, D = 700, 3, 128
    x = torch.randn(T, H, D, generator=g, device="cuda")
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    freqs = torch.from_numpy(moe.rope_freqs(D, 1e6)[0]).cuda()
    out = torch.empty_like(x)
    moe.rope(x, pos, freqs, T, H, D, out, interleaved=interleaved, dtype=0)
    y, _ = ref.rope(x, pos, freqs, D, interleaved, False, 1.0)
    a = pos.double()[:, None] * freqs
    c, s = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    u, v = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, 2)
    plain = (u * c - v * s, u * s + v * c)
    plain = torch.stack(plain, 3).flatten(2) if interleaved else torch.cat(plain, 2)
    assert float((out - y).norm()) <= 1.02 * float((plain - y).norm())
