"""Refusals of kvq_paged_decode_lse, kvq_attention_weights and kvq_evict_blocks (no
GPU): made-up pools and addresses, every call refused before it could launch."""
import ctypes

import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq
from paged_quantized_kv_kvq_gb300 import build as kbuild


@pytest.fixture(scope="module", autouse=True)
def L():
    kbuild.build()
    return kvq.lib()


def test_null_pools(L):
    assert L.kvq_paged_decode_lse(None, 16, 1, 1, 16, 1, 16, 1, 1.0, 16, 16, 16, 16, 0, None) == kvq.KVQ_ERR_INVALID_ARG
    assert L.kvq_attention_weights(None, 16, 1, 1, 16, 1, 16, 1, 1.0, 16, 1.0, None, 16, 1, None) == kvq.KVQ_ERR_INVALID_ARG
    assert L.kvq_evict_blocks(None, 16, 1, 1, 16, 1, 16, 1, 1, 0, 1, 16, 16, None, None, 0, None) == kvq.KVQ_ERR_INVALID_ARG


class FakePool:
    """The head of a kvq_pool (its PoolView): enough for the argument checks."""

    def __init__(self, bs=16, hkv=2, d=64):
        fields = [ctypes.c_void_p] * 4 + [ctypes.c_int64] + [ctypes.c_int] * 10

        class View(ctypes.Structure):
            _fields_ = [("f%d" % i, t) for i, t in enumerate(fields)]

        self.view = View()
        self.view.f4 = 100  # num_blocks
        for i, v in enumerate((bs, hkv, d, kvq.KVQ_FP16, 0, 1, 2)):
            setattr(self.view, "f%d" % (5 + i), v)
        self.room = ctypes.create_string_buffer(bytes(self.view), 4096)
        self.ptr = ctypes.cast(self.room, ctypes.c_void_p)


def _weights(L, pool, **kw):
    a = dict(q=16, S=1, hq=4, table=16, mb=10, lens=16, mc=100, scale=1.0, lse=16, decay=1.0, prev=None, scores=16, stride=100)
    a.update(kw)
    return L.kvq_attention_weights(pool.ptr, a["q"], a["S"], a["hq"], a["table"], a["mb"], a["lens"], a["mc"], a["scale"], a["lse"],
                                   a["decay"], a["prev"], a["scores"], a["stride"], None)


@pytest.mark.parametrize("kw", [dict(S=-1), dict(hq=0), dict(hq=3), dict(mb=0), dict(mc=-1), dict(stride=99), dict(mc=161, stride=200),
                                dict(scale=float("nan")), dict(decay=float("nan")), dict(q=None), dict(table=None), dict(lens=None),
                                dict(lse=None), dict(scores=None), dict(q=8)])
def test_weights_refusals(L, kw):
    assert _weights(L, FakePool(), **kw) == kvq.KVQ_ERR_INVALID_ARG


@pytest.mark.parametrize("decay", [float("inf"), float("-inf")])
def test_weights_need_a_finite_decay(L, decay):
    assert _weights(L, FakePool(), decay=decay) == kvq.KVQ_ERR_INVALID_ARG


def test_weights_of_the_longest_contexts(L):
    n = 2 ** 31 - 1
    assert _weights(L, FakePool(bs=64), mb=n // 64 + 1, mc=n, stride=n) == kvq.KVQ_ERR_UNSUPPORTED


def test_weights_nothing_to_do(L):
    assert _weights(L, FakePool(), S=0) == kvq.KVQ_OK
    assert _weights(L, FakePool(), mc=0, stride=0) == kvq.KVQ_OK


def _evict(L, pool, **kw):
    a = dict(scores=16, stride=160, S=1, table=16, mb=10, lens=16, mc=160, budget=4, sink=1, recent=2, to=16, lo=16, kept=None,
             so=None, os=0)
    a.update(kw)
    return L.kvq_evict_blocks(pool.ptr, a["scores"], a["stride"], a["S"], a["table"], a["mb"], a["lens"], a["mc"], a["budget"],
                              a["sink"], a["recent"], a["to"], a["lo"], a["kept"], a["so"], a["os"], None)


@pytest.mark.parametrize("kw", [dict(S=-1), dict(mb=0), dict(mc=-1), dict(stride=159), dict(mc=161, stride=170), dict(budget=0),
                                dict(budget=2), dict(sink=-1), dict(recent=0), dict(sink=2 ** 31 - 1), dict(scores=None),
                                dict(table=None), dict(lens=None), dict(to=None), dict(lo=None), dict(so=32, os=63), dict(so=16, os=64)])
def test_evict_refusals(L, kw):
    assert _evict(L, FakePool(), **kw) == kvq.KVQ_ERR_INVALID_ARG


def test_evict_too_long_and_nothing_to_do(L):
    n = 28673
    assert _evict(L, FakePool(bs=8), mb=n, mc=8 * n, stride=8 * n) == kvq.KVQ_ERR_UNSUPPORTED
    assert _evict(L, FakePool(), S=0) == kvq.KVQ_OK


def test_binding_checks():
    q = torch.zeros((2, 4, 64), dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros((2, 4), dtype=torch.int32)
    f = torch.zeros((2, 4))
    with pytest.raises(ValueError):
        kvq.kvq_paged_decode_lse(None, q, table, i, 4, 1.0, q, torch.zeros((2, 3)))
    with pytest.raises(ValueError):
        kvq.kvq_attention_weights(None, q, table, i, 4, 1.0, f, torch.zeros((2, 64)))
    with pytest.raises(ValueError):
        kvq.kvq_attention_weights(None, q, table, i, 4, 1.0, f, torch.zeros((2, 2, 64)), torch.zeros((2, 2, 63)))
    w = torch.zeros((2, 2, 64))
    with pytest.raises(ValueError):
        kvq.kvq_evict_blocks(None, w, table[:1], i, 4, 2, 0, 1, table, i)
    with pytest.raises(ValueError):
        kvq.kvq_evict_blocks(None, w, table, i, 4, 2, 0, 1, table[:, :2], i)
    with pytest.raises(ValueError):
        kvq.kvq_evict_blocks(None, w, table, i, 4, 2, 0, 1, table, i, kept=table)
    with pytest.raises(ValueError):
        kvq.kvq_evict_blocks(None, w, table, i, 4, 2, 0, 1, table, i, scores_out=w[:, :1])
