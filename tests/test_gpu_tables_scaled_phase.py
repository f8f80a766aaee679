"""build_tables_scaled against the rules in 60 decimal digits, at positions where a frequency of 53 bits is too little.

Bound, as the header has it: 6 * 2^-24 of the value (the two roundings of the rest of a phase, the series', the factor's
and its product's), and p 2^-65 + 2^-57 turns for the phase; beside these, the reference's own last step in 64 bits."""
import math
from decimal import Decimal, localcontext

import pytest
import torch

from gpu_util import lib, require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def turns(kind, rd, factor, original, theta):
    """Turns per position of every pair."""
    f, theta_, one = Decimal(factor), Decimal(theta), Decimal(1)
    low, high = (1, 32) if kind == "yarn" else (1, 4)
    w = [theta_ ** (Decimal(-2 * i) / rd) for i in range(rd // 2)]
    if kind == "linear":
        w = [x / f for x in w]
    elif kind == "ntk":
        base = theta_ * f ** (Decimal(rd) / (rd - 2))
        w = [base ** (Decimal(-2 * i) / rd) for i in range(rd // 2)]
    elif kind == "smooth":
        m = [min(max((original * x / TWO_PI - low) / (high - low), Decimal(0)), one) for x in w]
        w = [(1 - m) * x / f + m * x for x, m in zip(w, m)]
    else:
        pair = lambda n: rd * math.log(original / (n * 2 * math.pi)) / (2 * math.log(theta))
        a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rd - 1)
        m = [min(max(Decimal(i - a) / (b - a), Decimal(0)), one) for i in range(rd // 2)]
        w = [x / f * m + x * (1 - m) for x, m in zip(w, m)]
    return [x / TWO_PI for x in w], (0.1 * math.log(factor) + 1.0 if kind == "yarn" else 1.0)


@pytest.mark.parametrize("kind", ["linear", "ntk", "smooth", "yarn"])
@pytest.mark.parametrize("rd,theta", [(128, 5e5), (64, 1e4), (96, 1e6)])
@pytest.mark.parametrize("offset", [0, 10 ** 8, (1 << 31) - 40])
def test_phases(kind, rd, theta, offset):
    require_gpu()
    R = lib()
    rows = 24
    cos, sin = R.build_tables_scaled(kind, rd, rows, 8.0, 8192, theta=theta, pos_offset=offset)
    with localcontext() as context:
        context.prec = 60
        t, scale = turns(kind, rd, 8.0, 8192, theta)
        angle = torch.tensor([[float(x * p % 1 * TWO_PI) for x in t] for p in range(offset, offset + rows)], dtype=torch.float64)
    p = torch.arange(offset, offset + rows, dtype=torch.float64)[:, None]
    off = scale * (2 * math.pi * (p * 2.0 ** -65 + 2.0 ** -57) + 2.0 ** -50)
    for got, want in ((cos, scale * angle.cos()), (sin, scale * angle.sin())):
        d = (got.cpu().double() - want).abs()
        bound = 6 * U * want.abs() + off
        assert (d <= bound).all(), "%.2f of the bound" % (d / bound).max()


@pytest.mark.parametrize("low,high", [(1e-300, 2e-300), (5e-324, 1e-323), (1.0, math.nextafter(1.0, 2.0)), (1e300, 1.7e308)])
def test_ramps_of_any_width(low, high):
    """Pairs beyond the ramp, however narrow or far it is, are the unscaled ones, or those of every position divided."""
    require_gpu()
    R = lib()
    got = R.build_tables_scaled("smooth", 64, 40, 8.0, 4096, low_turns=low, high_turns=high, pos_offset=5)
    kept = R.build_tables_scaled("linear", 64, 40, 1.0, pos_offset=5)
    slowed = R.build_tables_scaled("linear", 64, 40, 8.0, pos_offset=5)
    n = 4096 * 1e4 ** (-torch.arange(32, dtype=torch.float64) / 32) / (2 * math.pi)
    for a, b, c in zip(got, kept, slowed):
        assert torch.equal(a.cpu(), torch.where(n > high, b.cpu(), c.cpu()))
