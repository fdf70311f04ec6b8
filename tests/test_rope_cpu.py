"""Host side of the rotation (no GPU): plans against exact integers, and every
refusal of kvq_rope_init, kvq_rope, kvq_rope_append and kvq_read_values."""
import ctypes
import math

import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq
from cache_ops_ref import angles, fractions, frequencies
from paged_quantized_kv_kvq_gb300 import build as kbuild


@pytest.fixture(scope="module", autouse=True)
def L():
    kbuild.build()
    return kvq.lib()


KW = {0: {}, 1: dict(factor=2.5), 2: dict(factor=8.0), 3: dict(factor=16.0, orig_len=4096.0, low=1.0, high=32.0),
      4: dict(factor=8.0, orig_len=8192.0, low=1.0, high=4.0)}


@pytest.mark.parametrize("scaling", list(KW))
@pytest.mark.parametrize("r", [16, 64, 112, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_plan(scaling, r, base):
    plan = kvq.kvq_rope_init(r, True, scaling, base=base, **KW[scaling])
    assert (plan.rotary_dim, plan.layout) == (r, kvq.KVQ_ROPE_INTERLEAVED)
    want = 0.1 * math.log(16.0) + 1 if scaling == 3 else 1.0
    assert abs(plan.magnitude - want) < 1e-6
    for got, f in zip(plan.turns, fractions(frequencies(r, base, scaling, **KW[scaling]))):
        assert abs(got - f) <= f * 2.0 ** -48  # a few roundings of pow and log
    assert not any(plan.turns[r // 2:])


def test_magnitude_is_taken():
    assert kvq.kvq_rope_init(64, scaling=3, magnitude=1.25, **KW[3]).magnitude == 1.25


def test_reference_angles_agree_with_floats():
    f = frequencies(64)
    a = angles(f, [0, 1, 100, -3])
    for t, p in enumerate((0, 1, 100, -3)):
        for j, w in enumerate(f):
            assert abs(math.cos(a[t, j]) - math.cos(p * w)) < 1e-12


@pytest.mark.parametrize("kw,status", [
    (dict(rotary_dim=0), kvq.KVQ_ERR_INVALID_ARG), (dict(rotary_dim=130), kvq.KVQ_ERR_INVALID_ARG),
    (dict(rotary_dim=31), kvq.KVQ_ERR_INVALID_ARG), (dict(rotary_dim=24), kvq.KVQ_ERR_UNSUPPORTED),
    (dict(rotary_dim=-16), kvq.KVQ_ERR_INVALID_ARG), (dict(scaling=5), kvq.KVQ_ERR_INVALID_ARG),
    (dict(scaling=-1), kvq.KVQ_ERR_INVALID_ARG), (dict(base=1.0), kvq.KVQ_ERR_INVALID_ARG),
    (dict(base=float("nan")), kvq.KVQ_ERR_INVALID_ARG), (dict(base=float("inf")), kvq.KVQ_ERR_INVALID_ARG),
    (dict(scaling=1, factor=0.5), kvq.KVQ_ERR_INVALID_ARG), (dict(scaling=1, factor=float("nan")), kvq.KVQ_ERR_INVALID_ARG),
    (dict(scaling=3, factor=2.0), kvq.KVQ_ERR_INVALID_ARG),
    (dict(scaling=3, factor=2.0, orig_len=100.0, low=4.0, high=4.0), kvq.KVQ_ERR_INVALID_ARG),
    (dict(scaling=4, factor=2.0, orig_len=100.0, low=0.0, high=4.0), kvq.KVQ_ERR_INVALID_ARG),
    (dict(scaling=2, factor=1e300), kvq.KVQ_ERR_INVALID_ARG),
    (dict(magnitude=-1.0), kvq.KVQ_ERR_INVALID_ARG), (dict(magnitude=float("nan")), kvq.KVQ_ERR_INVALID_ARG)])
def test_init_refusals(kw, status):
    with pytest.raises(kvq.KVQError) as e:
        kvq.kvq_rope_init(**{"rotary_dim": 64, **kw})
    assert e.value.status == status


def test_magnitude_must_fit_fp32():
    with pytest.raises(kvq.KVQError) as e:
        kvq.kvq_rope_init(64, magnitude=1e39)
    assert e.value.status == kvq.KVQ_ERR_INVALID_ARG
    assert kvq.kvq_rope_init(64, magnitude=1e38).magnitude == ctypes.c_float(1e38).value


def test_too_many_rows(L):
    """Rows that would need more than 2^31 - 1 CTAs."""
    assert _rope(L, hq=8192, qs=8192 * 128, qos=8192 * 128, T=(1 << 31) - 1) == kvq.KVQ_ERR_UNSUPPORTED


def test_null_plan_arguments(L):
    plan = kvq.RopePlan()
    assert L.kvq_rope_init(None, ctypes.byref(plan)) == kvq.KVQ_ERR_INVALID_ARG
    assert L.kvq_rope_init(ctypes.byref(kvq._RopeConfig()), None) == kvq.KVQ_ERR_INVALID_ARG
    cfg = kvq._RopeConfig(64, 2, 0, 10000.0, 1.0, 0.0, 0.0, 0.0, 0.0)
    assert L.kvq_rope_init(ctypes.byref(cfg), ctypes.byref(plan)) == kvq.KVQ_ERR_INVALID_ARG


def _rope(L, plan=None, x_type=0, q=16, qs=128, hq=1, k=16, ks=128, hk=1, d=128, pos=16, T=1, eps=0.0, qo=16, qos=128,
          ko=16, kos=128):
    """The C call with made-up addresses: every call here is refused before it could launch."""
    p = None if plan is None else ctypes.byref(plan)
    return L.kvq_rope(p, x_type, q, qs, hq, k, ks, hk, d, pos, T, None, None, eps, qo, qos, ko, kos, None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(hq=-1), dict(hk=-1), dict(d=0), dict(x_type=2), dict(x_type=-1), dict(eps=-1.0),
                                dict(eps=float("nan")), dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(q=8),
                                dict(k=24), dict(qo=2), dict(ko=8), dict(qs=127), dict(qs=132), dict(ks=64), dict(qos=120),
                                dict(kos=133)])
def test_rope_invalid_arguments(L, kw):
    assert _rope(L, **kw) == kvq.KVQ_ERR_INVALID_ARG


def test_rope_plan_checks(L):
    plan = kvq.kvq_rope_init(128)
    assert _rope(L, plan=plan, pos=None) == kvq.KVQ_ERR_INVALID_ARG
    assert _rope(L, plan=plan, d=64) == kvq.KVQ_ERR_INVALID_ARG  # more rotated channels than the head has
    for field, bad in (("rotary_dim", 8), ("rotary_dim", 40), ("rotary_dim", 144), ("layout", 7)):
        plan = kvq.kvq_rope_init(64)
        setattr(plan, field, bad)
        assert _rope(L, plan=plan) == kvq.KVQ_ERR_INVALID_ARG
    assert _rope(L, d=256) == kvq.KVQ_ERR_UNSUPPORTED
    assert _rope(L, T=1 << 31) == kvq.KVQ_ERR_UNSUPPORTED
    assert _rope(L, T=0) == kvq.KVQ_OK
    assert _rope(L, hq=0, hk=0) == kvq.KVQ_OK


def test_null_pools(L):
    assert L.kvq_rope_append(None, None, 0, None, 0, 0, None, 0, None, 0, None, None, 1, None, None, 0.0, None, 0,
                             None) == kvq.KVQ_ERR_INVALID_ARG
    assert L.kvq_read_values(None, None, 1, None, None, None) == kvq.KVQ_ERR_INVALID_ARG


def test_binding_checks():
    h = torch.zeros((2, 3, 64), dtype=torch.float16)
    plan = kvq.kvq_rope_init(64)
    with pytest.raises(ValueError):
        kvq.kvq_rope(plan, None, None, None)
    with pytest.raises(ValueError):
        kvq.kvq_rope(plan, h.float(), None, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):  # host rows
        kvq.kvq_rope(plan, h, None, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        kvq.kvq_rope_append(None, plan, None, h, h[:1], None, torch.zeros(2, dtype=torch.int64))


def test_block_format_layout():
    for fmt in kvq.BLOCK_FORMATS:
        lay = kvq.kvq_pool_layout_query(10, 16, 2, 128, fmt)
        assert lay["code_bytes"] == 2 * 10 * 16 * 2 * 128
        assert lay["scale_bytes"] == 10 * 2 * 16
        assert lay["page_bytes"] == 2 * 16 * 128 + 16
        assert kvq.kvq_pool_bytes(10, 8, 2, 64, fmt) > 0
