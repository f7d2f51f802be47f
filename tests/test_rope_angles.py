"""The angles of the rotary positions against 60-digit arithmetic that shares nothing with the library's float64."""
import decimal
from decimal import Decimal

import pytest
import torch

import paged_util as pu
import transformer_self_attention_gb300 as tsa

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
SCALINGS = [dict(), dict(base=500000.0), dict(scaling="linear", factor=3.7), dict(scaling="ntk", factor=7.3),
            dict(scaling="yarn", factor=5.3, original_len=4096)]


def _turns(rot, base=10000.0, scaling="none", factor=1.0, original_len=0):
    """Turns per position of the pairs (Decimal), by the definition."""
    base, factor = Decimal(base), Decimal(factor)
    if scaling == "ntk":
        base *= (factor.ln() * rot / (rot - 2)).exp()
    out = []
    for p in range(rot // 2):
        f = (base.ln() * (-2 * p) / rot).exp()
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            g = min(Decimal(1), max(Decimal(0), (original_len * f / (2 * PI) - 1) / 31))
            f = f * g + f / factor * (1 - g)
        out.append(f / (2 * PI))
    return out


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("rot", [4, 26, 128, 256])
def test_frequencies_are_within_their_bound(rot, kw):
    """2^-53 turns a position, of which the frequency's own error may take 0.78: the quotient by 2 pi takes the rest, f
    / (2 pi) (2^-54 + 2^-53) at most, f <= 1."""
    with decimal.localcontext() as c:
        c.prec = 60
        f, _ = tsa.RotaryPositions(256, rot, **kw).frequencies()
        for got, want in zip(f.tolist(), _turns(rot, **kw)):
            assert abs(Decimal(got) / (2 * PI) - want) <= Decimal(2) ** -53 * Decimal("0.78")


@pytest.mark.gpu
@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions(layout, kw):
    """Elements at positions to 2^31: the float32 bound of a rotated element, and 2 pi 2^-53 rad a position."""
    d, pos = 128, [0, 1, -5, 4095, (1 << 20) + 3, (1 << 24) + 1, -(1 << 27) - 9, 2 ** 31 - 1, -2 ** 31]
    x = torch.randn((1, 2, len(pos), d), generator=torch.Generator().manual_seed(1))
    rope = tsa.RotaryPositions(d, layout=layout, **kw)
    y = rope(x.cuda(), positions=torch.tensor(pos, dtype=torch.int32).cuda()).double().cpu()
    _, amp = rope.frequencies()
    i = torch.arange(d // 2)
    first, second = (i, i + d // 2) if layout == "half" else (2 * i, 2 * i + 1)
    with decimal.localcontext() as c:
        c.prec = 60
        turns = _turns(d, **kw)
        angles = [[float((t * n) % 1 * 2 * PI) for t in turns] for n in pos]
    angle = torch.tensor(angles, dtype=torch.float64)
    a, b = x.double()[..., first], x.double()[..., second]
    want, size = torch.empty_like(y), torch.empty_like(y)
    want[..., first] = (a * torch.cos(angle) - b * torch.sin(angle)) * amp
    want[..., second] = (a * torch.sin(angle) + b * torch.cos(angle)) * amp
    size[..., first] = size[..., second] = (a.abs() + b.abs()) * amp
    far = torch.tensor(pos, dtype=torch.float64).abs()[:, None] * (2 * float(PI) * 2.0 ** -53)
    assert float(((y - want).abs() - pu.rope_bound(want, size, torch.float32) - size * far).max()) <= 0


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_cosines_and_sines_are_float32_ones(layout):
    """Rows of pairs (1, 0) come back as (cos t, sin t).  Each is off by an ulp at most (CUDA's bound for sincospif; an ulp
    is at most 2^-23 of the number) and by the angle's own error times the other one: t is brought to at most an eighth of
    a turn exactly, a float32 number of half turns there is rounded by 2^-27 and cut by 2^-33 of one, and the frequencies
    (theirs and the reference's) and the reference's product add less than 1e-11 rad at these positions."""
    d, S = 256, 4096
    x = torch.zeros((1, 1, S, d))
    i = torch.arange(d // 2)
    first, second = (i, i + d // 2) if layout == "half" else (2 * i, 2 * i + 1)
    x[..., first] = 1.0
    y = tsa.RotaryPositions(d, layout=layout)(x.cuda()).double().cpu()[0, 0]
    f, _ = pu.frequencies(d)
    t = torch.arange(S, dtype=torch.float64)[:, None] * f
    cos, sin = torch.cos(t), torch.sin(t)
    turn = float(PI) * (2.0 ** -27 + 2.0 ** -33) + 1e-11
    for got, want, other in ((y[:, first], cos, sin), (y[:, second], sin, cos)):
        assert float(((got - want).abs() - other.abs() * turn - want.abs() * 2.0 ** -23).max()) <= 0
