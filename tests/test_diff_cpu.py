"""Differential attention without a GPU: what the calls refuse, in C and in the binding."""
import ctypes

import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq
from paged_quantized_kv_kvq_gb300 import build as kbuild

BS, HKV, D = 16, 2, 128
HANDLE = kvq.PoolHandle(0)
HANDLE.shape = (BS, HKV, D)


def _half(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _args(**kw):
    a = dict(q=_half(3, 4, D), block_table=_i(3, 6), context_lens=_i(3), max_context_len=96, sm_scale=0.125, lam=torch.zeros(4),
             out=_half(3, 4, D))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,match", [
    (dict(q=_half(3, 4, 64), out=_half(3, 4, 64)), "head_dim of 128"), (dict(q=_half(3, 3, D), out=_half(3, 3, D), lam=torch.zeros(3)), "multiple of its 2"),
    (dict(block_table=_i(2, 6)), "block_table"), (dict(context_lens=_i(2)), "context_lens"), (dict(lam=torch.zeros(8)), "lam must"),
    (dict(out=_half(3, 8, D)), "out must"), (dict(q=_half(12, D)), "q must"), (dict(norm_weight=torch.zeros(64)), "norm_weight"),
    (dict(), "CUDA device")])
def test_decode_shapes(kw, match):
    with pytest.raises(ValueError, match=match):
        kvq.kvq_diff_decode(HANDLE, **_args(**kw))


@pytest.mark.parametrize("kw,match", [
    (dict(q=_half(3, 4, 64), out=_half(3, 4, 64)), "head_dim of 128"), (dict(q_start=_i(3)), "q_start"), (dict(block_table=_i(2, 6)), "block_table"),
    (dict(lam=torch.zeros(2)), "lam must"), (dict(out=_half(2, 4, D)), "out must"), (dict(), "CUDA device")])
def test_prefill_shapes(kw, match):
    with pytest.raises(ValueError, match=match):
        kvq.kvq_diff_prefill(HANDLE, **_args(max_q_len=1, workspace=None, **{"q_start": _i(4), **kw}))


def test_c_refusals():
    kbuild.build()
    L = kvq.lib()
    x = ctypes.c_void_p(4096)
    assert L.kvq_diff_decode(None, x, 1, 2, x, 1, x, 1, 1.0, x, None, 0.0, 1.0, x, None, 0, None) == kvq.KVQ_ERR_INVALID_ARG
    assert L.kvq_diff_prefill(None, x, 1, 1, 2, x, 1, x, 1, x, 1, 1.0, x, None, 0.0, 1.0, x, None, 0, None) == kvq.KVQ_ERR_INVALID_ARG
    assert L.kvq_diff_decode_workspace_bytes(None, 1, 2, 16) == 0
    assert L.kvq_diff_prefill_workspace_bytes(None, 1, 1, 2, 16) == 0
