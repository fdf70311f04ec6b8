"""Equal maps at lambda 1 leave rows of zeros, which a norm without eps keeps."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq
from cache_ops_ref import tokens
from test_gpu_diff import FORMATS, _filled, _t

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
def test_equal_maps_cancel(fmt, group, d):
    """Both halves of every query and key alike: decode whole and cut over many warps, prompts."""
    if group > d // 2:
        pytest.skip("a scale group spans both halves")
    bs, H, hkv = 16, 4, 2
    pool, _, table, lens, rng = _filled(fmt, group, bs, hkv, d, [40, 3000, 9, 200], seed=d)
    slots = np.concatenate([tokens(table, lens, s, bs) for s in range(4)])
    k, v = (rng.standard_normal((len(slots), hkv, d)).astype(np.float16) for _ in range(2))
    k[..., d // 2:] = k[..., :d // 2]
    if fmt == kvq.KVQ_INT8_PER_CHANNEL:
        kvq.kvq_calibrate_channel_scales(pool.handle, _t(k), _t(v))
    pool.append(_t(k), _t(v), _t(slots))
    n = [40, 70, 9, 200]
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q = rng.standard_normal((start[-1], H, d)).astype(np.float16)
    q[..., d // 2:] = q[..., :d // 2]
    lam = np.array([1, 1, 0.5, 1], np.float32)
    w = _t(rng.uniform(0.5, 1.5, d).astype(np.float32))
    for weight in (None, w):
        out = pool.diff_decode(_t(q[start[1:] - 1]), _t(table), _t(lens), 3000, _t(lam), weight, 0.0)
        pre = pool.diff_prefill(_t(q), _t(start), 200, _t(table), _t(lens), 3000, _t(lam), weight, 0.0)
        assert pool.error() == kvq.KVQ_OK
        for x in (out, pre):
            assert (x[:, [0, 1, 3]] == 0).all(), x[:, [0, 1, 3]].abs().max()
            assert torch.isfinite(x).all() and (x[:, 2] != 0).any(-1).all()
    pool.close()
