"""The angle of the rotary positions, where its last bits show: sines near half
turns and cosines near quarter turns, against integer arithmetic.

With x_a = 1, x_b = 0 and scale 1 the results are the cosine and the sine.  The
angle is off by 2^-32 of a turn, and the frequency in turns, a product of two fp64
numbers one of which is 1 / (2 pi) rounded, by 2^-52 of its size, times the
position.  The value itself, small there, is off by a few steps: 2^-22 of it.
"""
import math

import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu

PI = 314159265358979323846264338327950288419716939937510582097494459  # times 10^62
BITS = 160


def turns(f):
    """f radians in turns, times 2^BITS (f: a float, exactly)."""
    a, b = f.as_integer_ratio()
    return (a * 10 ** 62 << BITS) // (2 * PI * b)


@pytest.mark.parametrize("rot", [2, 8])          # narrow and 16-byte accesses
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("f", [1.0, 0.7310585786300049])
def test_near_quarter_turns(rot, interleaved, f):
    import long_context_attention_causal_gb300 as pa
    unit, one = turns(f), 1 << BITS
    near = one >> 13
    found = []                                   # (position, quarter turns, the rest)
    for p in range(-(1 << 19), 1 << 19, 7):
        t = p * unit % one
        quarters = (4 * t + (one >> 1)) // one   # nearest
        rest = t - quarters * (one >> 2)
        if abs(rest) < near:
            found.append((p, quarters % 4, rest))
    assert len(found) > 100 and {n for _, n, _ in found} == {0, 1, 2, 3}
    N, half = len(found), rot // 2
    x = torch.zeros((N, 1, 64), device=dev())
    if interleaved:
        x[..., 0:rot:2] = 1.0
    else:
        x[..., :half] = 1.0
    pos = torch.tensor([p for p, _, _ in found], dtype=torch.int32, device=dev())
    freq = torch.full((half,), f, dtype=torch.float64, device=dev())
    y, _ = pa.rope(x, None, pos, freq, interleaved=interleaved)
    y = y[:, 0].double().cpu()
    cos, sin = (y[:, 0:rot:2], y[:, 1:rot:2]) if interleaved else (y[:, :half], y[:, half:rot])
    for i, (p, n, rest) in enumerate(found):
        small = math.sin(2.0 * math.pi * (rest / one))
        # sin(n / 4 + r) = sin r, cos r, -sin r, -cos r;  cos = cos r, -sin r, ...
        got = (sin, cos, sin, cos)[n][i]
        want = (small, -small, -small, small)[n]
        tol = 2.0 * math.pi * 2.0 ** -32 + abs(p) * f * 2.0 ** -52 + 2.0 ** -22 * abs(want)
        assert ((got - want).abs() <= tol).all(), (p, n, want, got)
        large = (cos, sin, cos, sin)[n][i]
        assert ((large - (1.0, 1.0, -1.0, -1.0)[n] * math.cos(2.0 * math.pi * (rest / one))).abs()
                <= 2.0 ** -22).all()
