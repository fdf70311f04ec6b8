"""Block bookkeeping without a GPU: what the calls refuse, in C and in the binding."""
import ctypes

import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq
from paged_quantized_kv_kvq_gb300 import build as kbuild

HANDLE = kvq.PoolHandle(0)
HANDLE.shape = (16, 2, 128)


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kvq.lib()


def _i(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


def _extend(**kw):
    a = dict(new_tokens=_i(3), block_table=_i(3, 6), context_lens=_i(3), free_list=_i(9), free_count=_i(1), lens_out=_i(3),
             count_out=_i(1), q_start=_i(4), slot_mapping=_i(20, dtype=torch.int64), positions=_i(20, dtype=torch.int64))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,match", [
    (dict(new_tokens=_i(2)), "new_tokens"), (dict(block_table=_i(2, 6)), "block_table"), (dict(block_table=_i(18)), "block_table"),
    (dict(lens_out=_i(4)), "new_tokens"), (dict(q_start=_i(3)), "q_start"), (dict(positions=_i(19, dtype=torch.int64)), "positions"),
    (dict(), "CUDA device")])
def test_extend_shapes(kw, match):
    with pytest.raises(ValueError, match=match):
        kvq.kvq_extend_tables(HANDLE, **_extend(**kw))


@pytest.mark.parametrize("kw,match", [
    (dict(block_table=_i(2, 6)), "block_table"), (dict(new_lens=_i(2)), "block_table"), (dict(), "CUDA device")])
def test_release_shapes(kw, match):
    a = dict(block_table=_i(3, 6), old_lens=_i(3), new_lens=_i(3), free_list=_i(9), free_count=_i(1), count_out=_i(1))
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        kvq.kvq_release_blocks(HANDLE, **a)


class _FakePool(ctypes.Structure):
    """Stands for a pool whose handle the checks look into no further than its view."""

    _fields_ = [("bytes", ctypes.c_char * 512)]


def test_c_refusals(L):
    p = ctypes.cast(ctypes.pointer(_FakePool()), ctypes.c_void_p)
    x = ctypes.c_void_p(4096)  # never looked at: every call here is refused first
    extend = lambda pool=p, n=x, S=1, t=x, mb=4, lens=x, fl=x, cap=8, fc=x, lo=x, co=x, qs=x, sm=x, po=x, T=8: L.kvq_extend_tables(  # noqa: E731
        pool, n, S, t, mb, lens, fl, cap, fc, lo, co, qs, sm, po, T, None)
    bad = kvq.KVQ_ERR_INVALID_ARG
    for kw in (dict(pool=None), dict(S=-1), dict(mb=0), dict(cap=-1), dict(T=-1), dict(n=None), dict(t=None), dict(lens=None),
               dict(fl=None), dict(fc=None), dict(lo=None), dict(co=None), dict(qs=None), dict(sm=None), dict(po=None)):
        assert extend(**kw) == bad, kw
    for kw in (dict(S=16385), dict(cap=0x7fffffff), dict(T=0x7fffffff)):
        assert extend(**kw) == kvq.KVQ_ERR_UNSUPPORTED, kw
    release = lambda pool=p, t=x, mb=4, a=x, b=x, S=1, sh=0, fl=x, cap=8, fc=x, co=x: L.kvq_release_blocks(  # noqa: E731
        pool, t, mb, a, b, S, sh, fl, cap, fc, co, None)
    for kw in (dict(pool=None), dict(t=None), dict(mb=0), dict(a=None), dict(b=None), dict(S=-1), dict(sh=-1), dict(fl=None),
               dict(cap=-1), dict(fc=None), dict(co=None)):
        assert release(**kw) == bad, kw
    assert release(S=16385) == kvq.KVQ_ERR_UNSUPPORTED
    assert release(S=16384, mb=1 << 17) == kvq.KVQ_ERR_UNSUPPORTED
