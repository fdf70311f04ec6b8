"""Prompts of a sequence whose length is below zero: no position is left for its rows, which get
zeros and are flagged, however close to -2^31 the length is (less the rows it wraps around)."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq
from test_gpu_diff import DEV, FORMATS, _filled, _t

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("least", [-2 ** 31, -2 ** 31 + 60, -1])
@pytest.mark.parametrize("fmt,group", FORMATS)
def test_negative_lengths(fmt, group, least):
    bs, hq, hkv, d = 16, 4, 2, 64 if 0 < group < 64 else 128
    pool, _, table, lens, rng = _filled(fmt, group, bs, hkv, d, [70, 100], seed=2)
    start = _t(np.array([0, 70, 140], np.int32))
    q = _t(rng.standard_normal((140, hq, d)).astype(np.float16))
    bad = lens.copy()
    bad[0] = least
    nb = kvq.kvq_prefill_workspace_bytes(pool.handle, 2, 100)
    ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=DEV)
    for two in (False, True):
        got = {}
        for x in (lens, bad):
            out = torch.full((140, hq, d), 7.0, device=DEV)
            if two:
                kvq.kvq_prefill_ex(pool.handle, q, start, 70, _t(table), _t(x), 100, d ** -0.5, out, ws if nb else None)
            else:
                kvq.kvq_prefill(pool.handle, q, start, 70, _t(table), _t(x), 100, d ** -0.5, out)
            assert pool.error() == (kvq.KVQ_OK if x is lens else kvq.KVQ_ERR_OUT_OF_RANGE)
            got[x is bad] = out
        assert (got[True][:70] == 0).all()
        assert torch.equal(got[True][70:], got[False][70:])
    lam = torch.rand(hq, device=DEV)
    out = pool.diff_prefill(q, start, 70, _t(table), _t(bad), 100, lam)
    assert pool.error() == kvq.KVQ_ERR_OUT_OF_RANGE
    assert (out[:70] == 0).all() and (out[70:] != 0).any(-1).all()
    pool.close()
