"""Fractions of a rotation plan against frequencies of 60 digits (no GPU)."""
import math
from decimal import Decimal, getcontext

import pytest

import paged_quantized_kv_kvq_gb300 as kvq
from paged_quantized_kv_kvq_gb300 import build as kbuild

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def exact_turns(r, base, scaling=0, factor=1.0, orig_len=0.0, low=0.0, high=0.0):
    """Turns per position of each pair, by the definitions in kvq.h."""
    base, factor, n, low, high = (Decimal(x) for x in (base, factor, orig_len, low, high))
    if scaling == kvq.KVQ_ROPE_BASE:
        base *= (factor.ln() * r / (r - 2)).exp()
    ln = base.ln()
    if scaling == kvq.KVQ_ROPE_PARTS:
        lo, hi = (r * (n / (2 * PI * b)).ln() / (2 * ln) for b in (high, low))
        lo, hi = max(Decimal(math.floor(lo)), Decimal(0)), min(Decimal(math.ceil(hi)), Decimal(r - 1))
    out = []
    for i in range(r // 2):
        f, ramp = (-2 * i * ln / r).exp(), Decimal(0)
        if scaling == kvq.KVQ_ROPE_LINEAR:
            ramp = Decimal(1)
        elif scaling == kvq.KVQ_ROPE_PARTS:
            ramp = min(max((i - lo) / (hi - lo), Decimal(0)), Decimal(1))
        elif scaling == kvq.KVQ_ROPE_BANDS:
            ramp = 1 - min(max((n * f / (2 * PI) - low) / (high - low), Decimal(0)), Decimal(1))
        out.append((f * (1 - ramp) + f / factor * ramp) / (2 * PI))
    return out


def exact_angle(turns, pos):
    """pos * turns in radians, within half a turn."""
    t = turns * int(pos)
    t -= t.to_integral_value("ROUND_HALF_EVEN")
    return float(t * 2 * PI)


KW = [(0, {}), (1, dict(factor=2.5)), (2, dict(factor=8.0)), (2, dict(factor=1000.0)),
      (3, dict(factor=16.0, orig_len=4096.0, low=1.0, high=32.0)), (4, dict(factor=8.0, orig_len=8192.0, low=1.0, high=4.0)),
      (4, dict(factor=3.0, orig_len=131072.0, low=1.0, high=1000.0))]


@pytest.mark.parametrize("scaling,kw", KW)
@pytest.mark.parametrize("r", [16, 96, 128])
@pytest.mark.parametrize("base", [1.5, 10000.0, 500000.0, 1e8])
def test_fractions(scaling, kw, r, base):
    """Within 2^-52 of a turn: frequencies of at most 1 radian in fp64, where the power
    (2^-52 from itself, as much from a stretched base, 2^-54 from its exponent), the
    two roundings of f / 2 pi and four of the ramp are less than 6 * 2^-52 of f, over
    2 pi."""
    if scaling == 3 and base == 1.5:
        pytest.skip("the ramp's ends lie outside the pairs (tested on their own)")
    kbuild.build()
    plan = kvq.kvq_rope_init(r, scaling=scaling, base=base, **kw)
    for got, want in zip(plan.turns, exact_turns(r, base, scaling, **kw)):
        assert abs(got - want * 2 ** 64) <= 2 ** 12
