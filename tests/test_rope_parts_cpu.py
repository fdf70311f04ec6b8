"""The ramp of KVQ_ROPE_PARTS against its definition by turns, where the ends of the
ramp lie outside the pairs (no GPU)."""
import math

import pytest

import paged_quantized_kv_kvq_gb300 as kvq
from paged_quantized_kv_kvq_gb300 import build as kbuild


@pytest.fixture(scope="module", autouse=True)
def L():
    kbuild.build()
    return kvq.lib()


def _share(plan, base, factor, i):
    """How far pair i is divided: 0 not at all, 1 by the factor."""
    f = base ** (-2.0 * i / plan.rotary_dim)
    got = plan.turns[i] / 2.0 ** 64 * 2 * math.pi
    return (f - got) / (f - f / factor)


CASES = [(128, 10000.0, 4096.0, 1000.0, 2000.0), (64, 10000.0, 100.0, 32.0, 64.0), (128, 5.0, 8192.0, 1.0, 32.0),
         (64, 10000.0, 4.0, 1.0, 32.0), (16, 500000.0, 1.0, 0.5, 0.6), (32, 1.5, 1e6, 1.0, 2.0),
         (128, 10000.0, 8192.0, 1.0, 32.0), (128, 10000.0, 4096.0, 1.0, 32.0), (96, 500000.0, 8192.0, 1.0, 4.0),
         (64, 10000.0, 150.0, 1.0, 32.0), (128, 1.0001, 2 * math.pi, 0.9, 1.1)]


@pytest.mark.parametrize("r,base,n,low,high", CASES)
def test_pairs_beyond_the_ramp(r, base, n, low, high):
    """Above `high` turns nothing is divided, below `low` all of it, and the share never
    falls from a pair to the next; rounded outwards to whole pairs, the ramp may take in
    one pair beyond either end."""
    plan = kvq.kvq_rope_init(r, scaling=kvq.KVQ_ROPE_PARTS, base=base, factor=8.0, orig_len=n, low=low, high=high)
    turns = [n * base ** (-2.0 * i / r) / (2 * math.pi) for i in range(r // 2)]
    share = [_share(plan, base, 8.0, i) for i in range(r // 2)]
    for i, (t, s) in enumerate(zip(turns, share)):
        assert -1e-9 <= s <= 1 + 1e-9
        if t >= high and (i + 1 == len(turns) or turns[i + 1] >= high):
            assert abs(s) < 1e-9, i
        # (a ramp that would end behind the last channel ends there)
        if t <= low and (i == 0 or turns[i - 1] <= low):
            assert abs(s - 1) < 1e-9, i
        if i:
            assert s >= share[i - 1] - 1e-9


def test_crossed_ends():
    """All pairs slower than `low`: every one divided; all faster than `high`: none."""
    plan = kvq.kvq_rope_init(128, scaling=kvq.KVQ_ROPE_PARTS, factor=4.0, orig_len=4096.0, low=1000.0, high=2000.0)
    whole = kvq.kvq_rope_init(128, scaling=kvq.KVQ_ROPE_LINEAR, factor=4.0)
    assert all(abs(a - b) <= b * 2.0 ** -48 for a, b in zip(plan.turns, whole.turns))
    plan = kvq.kvq_rope_init(128, scaling=kvq.KVQ_ROPE_PARTS, base=5.0, factor=4.0, orig_len=8192.0, low=1.0, high=32.0)
    plain = kvq.kvq_rope_init(128, base=5.0)
    assert all(abs(a - b) <= b * 2.0 ** -48 for a, b in zip(plan.turns, plain.turns))
