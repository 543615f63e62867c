"""The table of rotary steps against frequencies in 60 decimal digits: a step is off by 2^-52 of a turn at most, 2^-51
for the blended scalings (the bounds that the header states for a position, at position 1)."""
from decimal import Decimal, getcontext

import numpy as np
import pytest

dlo = pytest.importorskip("layerwise_weight_offload_slot_gb300")

getcontext().prec = 60
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
FACTOR, LENGTH, FAST, SLOW = 8.0, 8192.0, 32.0, 1.0


def frequencies(dim, theta, scaling):
    """f of every pair of an axis, from the definitions."""
    theta, factor = Decimal(theta), Decimal(FACTOR)
    if scaling == dlo.ROPE_BASE and dim > 2:
        theta *= factor ** (Decimal(dim) / (dim - 2))
    pair = [dim * (Decimal(LENGTH) / (TWO_PI * Decimal(t))).ln() / (2 * theta.ln()) for t in (FAST, SLOW)]
    low, high = max(0, int(pair[0].to_integral_value("ROUND_FLOOR"))), min(dim - 1, int(pair[1].to_integral_value("ROUND_CEILING")))
    out = []
    for p in range(dim // 2):
        f = theta ** (Decimal(-2 * p) / dim)
        keep = Decimal(1)
        if scaling == dlo.ROPE_LINEAR:
            keep = Decimal(0)
        elif scaling == dlo.ROPE_BY_TURNS:
            keep = (Decimal(LENGTH) * f / TWO_PI - Decimal(SLOW)) / (Decimal(FAST) - Decimal(SLOW))
        elif scaling == dlo.ROPE_BY_INDEX:
            keep = 1 - (Decimal(p) - low) / max(Decimal(high - low), Decimal("0.001"))
        keep = min(Decimal(1), max(Decimal(0), keep))
        out.append(f * (keep + (1 - keep) / factor))
    return out


@pytest.mark.parametrize("scaling", range(5))
@pytest.mark.parametrize("dim", [2, 24, 64, 128, 254])
def test_steps(dim, scaling):
    for theta in (1.5, 100.0, 10000.0, 500000.0, 1e9):
        r = dlo.make_rope(heads=1, head_dim=256, ldx=256, ldy=256,
                          axes=[dict(dim=dim, theta=theta, scaling=scaling, factor=FACTOR, length=LENGTH, fast=FAST, slow=SLOW)])
        steps = dlo.dlo_rope_steps(r).view(np.uint64).tolist()
        bound = 2.0 ** (-52 if scaling < dlo.ROPE_BY_TURNS else -51)
        for p, (s, f) in enumerate(zip(steps, frequencies(dim, theta, scaling))):
            assert abs(float(Decimal(s) / 2 ** 64 - f / TWO_PI)) <= bound, (theta, p)
