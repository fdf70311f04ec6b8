"""Lengths below zero in a cascade: a sequence with such a length has nothing to attend, as one of
length zero, however close to -2^31 the length is (less the prefix it wraps around in 32 bits)."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq
from test_gpu_diff import FORMATS, _filled, _t

pytestmark = pytest.mark.gpu
LEAST = -2 ** 31


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("bs", [16, 64])
def test_negative_lengths(fmt, group, bs):
    hq, hkv, d, S = 8, 2, 64 if fmt == kvq.KVQ_FP16 or group < 64 else 128, 6
    pool, _, table, _, rng = _filled(fmt, group, bs, hkv, d, [4 * bs + 5] * S, seed=bs)
    table[:, :2] = table[0, :2]
    lens = np.array([LEAST, 4 * bs + 5, LEAST + 2 * bs - 1, -1, 3 * bs, LEAST + 1], np.int32)
    q = _t(rng.standard_normal((S, hq, d)).astype(np.float16))
    for prefix in (0, 1, 2):
        got = pool.cascade_decode(q, _t(table), _t(lens), 4 * bs + 5, prefix)
        want = pool.cascade_decode(q, _t(table), _t(np.maximum(lens, 0)), 4 * bs + 5, prefix)
        assert pool.error() == kvq.KVQ_OK
        assert torch.equal(got, want)
        assert (got[_t(lens) < 0] == 0).all() and (got[_t(lens) > 0] != 0).any(-1).all()
    pool.close()
