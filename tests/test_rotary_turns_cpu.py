"""The rotary table's 64-bit turns against 60 digits: each within 2 of its last place, so that the angle of a position is
off by at most 2^-63 turns times the position."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest

import precision_attention_nvfp4_b200 as fp

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module", autouse=True)
def lib():
    from precision_attention_nvfp4_b200 import build
    build.build()


def exact(dim, base, scaling, factor, length, fast, slow):
    """Turns a position of every pair."""
    base, factor, length, fast, slow = (Decimal(x) for x in (base, factor, length, fast, slow))
    if scaling == "ntk":
        base = base * factor ** (Decimal(dim) / (dim - 2))
    out = []
    if scaling == "yarn":
        at = lambda t: dim * (length / (2 * PI * t)).ln() / (2 * base.ln())  # noqa: E731
        lo, hi = max(0, math.floor(at(fast))), min(dim - 1, math.ceil(at(slow)))
    for i in range(dim // 2):
        f = base ** (Decimal(-2 * i) / dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            r = min(Decimal(1), max(Decimal(0), (i - lo) / max(Decimal(hi - lo), Decimal(0.001))))
            f = f * (1 - r) + f / factor * r
        elif scaling == "wavelength":
            k = min(Decimal(1), max(Decimal(0), (length * f / (2 * PI) - slow) / (fast - slow)))
            f = f * k + f / factor * (1 - k)
        out.append(f / (2 * PI))
    return out


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "wavelength"])
@pytest.mark.parametrize("dim,base,factor", [(128, 10000.0, 8.0), (64, 500000.0, 16.0), (48, 10000.0, 3.7), (16, 2.5, 1.0)])
def test_turns(scaling, dim, base, factor):
    fast = 32.0 if scaling == "yarn" else 4.0
    t = fp.rotary_table(dim, base=base, scaling=scaling, factor=factor, original_length=4096.0, device="cpu")
    want = exact(dim, base, scaling, factor, 4096.0, fast, 1.0)
    for got, w in zip(t.turns.numpy().view(np.uint64).tolist(), want):
        assert abs(Decimal(got) - w * 2 ** 64) <= 2, (got, w)
