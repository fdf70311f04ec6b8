"""Prompts at softmax scales of zero and below it, against float64, in every format."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq
from cache_ops_ref import attention, tokens
from test_gpu_diff import DEV, FORMATS, _filled, _t, diff_ref

pytestmark = pytest.mark.gpu
# Scores of up to 2^5 in magnitude and partial sums of twice that in powers of two, eight sums of the tensor core
# within 2^-23 of them: a weight within ln 2 * 2^-14 of itself at worst, and a result moves by that much of the
# values' spread, twice the largest value at most.
SPREAD = 2.0 ** -13


@pytest.mark.parametrize("scale", [0.0, -0.0, -0.125, -1.0, 0.3, 2.0 ** -149])
@pytest.mark.parametrize("fmt,group", FORMATS)
def test_prefill(fmt, group, scale):
    bs, hq, hkv, d = 16, 4, 2, 64 if group != 0 and group < 64 else 128
    pool, vals, table, lens, rng = _filled(fmt, group, bs, hkv, d, [150, 64, 7, 0], seed=5, fill_byte=0xFF if fmt == kvq.KVQ_FP4_E2M1 else 0)
    n = [150, 3, 7, 0]
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q = (0.25 * rng.standard_normal((start[-1], hq, d))).astype(np.float16)
    rows_lens = np.concatenate([np.arange(lens[s] - n[s], lens[s]) + 1 for s in range(4)]).astype(np.int32)
    seq = np.repeat(np.arange(4), n)
    want = attention(lambda r: vals[tokens(table[seq], rows_lens, r, bs)], q, rows_lens, scale)[0]
    for two in (False, True):
        got = torch.full((int(start[-1]), hq, d), 7.0, device=DEV)
        if two:
            nb = kvq.kvq_prefill_workspace_bytes(pool.handle, 4, 150)
            ws = torch.empty(nb, dtype=torch.uint8, device=DEV) if nb else None
            kvq.kvq_prefill_ex(pool.handle, _t(q), _t(start), 150, _t(table), _t(lens), 150, scale, got, ws)
        else:
            kvq.kvq_prefill(pool.handle, _t(q), _t(start), 150, _t(table), _t(lens), 150, scale, got)
        assert pool.error() == kvq.KVQ_OK
        np.testing.assert_allclose(got.cpu().numpy(), want, rtol=0, atol=SPREAD * np.abs(vals[:, 1]).max())
    # the same rows as single tokens
    last = start[1:4] - 1
    one = pool.decode(_t(q[last]), _t(table[:3]), _t(lens[:3]), 150, sm_scale=scale)
    np.testing.assert_allclose(one.cpu().numpy(), want[last], rtol=0, atol=SPREAD * np.abs(vals[:, 1]).max())
    pool.close()


@pytest.mark.parametrize("scale", [0.0, -0.3])
@pytest.mark.parametrize("fmt,group", FORMATS)
def test_differential_prefill(fmt, group, scale):
    bs, H, hkv, d = 16, 4, 2, 64 if group != 0 and group < 64 else 128
    pool, vals, table, lens, rng = _filled(fmt, group, bs, hkv, d, [150, 64], seed=6)
    n = [150, 3]
    start = np.array([0, 150, 153], np.int32)
    q = rng.standard_normal((153, H, d)).astype(np.float16)
    lam = np.array([0.4, 0.9, -0.2, 0.0], np.float32)
    rows_lens = np.concatenate([np.arange(lens[s] - n[s], lens[s]) + 1 for s in range(2)]).astype(np.int32)
    seq = np.repeat(np.arange(2), n)
    want, maps = diff_ref(lambda r: vals[tokens(table[seq], rows_lens, r, bs)], q, rows_lens, lam.astype(np.float64), None, 0.0, 1.0, scale)
    out = pool.diff_prefill(_t(q), _t(start), 150, _t(table), _t(lens), 150, _t(lam), sm_scale=scale)
    assert pool.error() == kvq.KVQ_OK
    # a map is a mean of values, within SPREAD of their largest; half an fp16 step
    got = out.cpu().numpy().astype(np.float64)
    bound = np.abs(want) * 2.0 ** -11 + (1 + np.abs(lam))[None, :, None] * SPREAD * np.abs(vals[:, 1]).max()
    assert (np.abs(got - want) <= bound).all(), np.abs(got - want).max()
    pool.close()
