"""The cascade over 4-bit floats held to the bound of the other ways to attend (its weights and
sums are those of the decode: two fp16 parts, fp32)."""
import numpy as np
import pytest

import paged_quantized_kv_kvq_gb300 as kvq
from test_gpu_fp4 import _filled, _near, _t

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs,hq,hkv,d", [(16, 8, 2, 128), (32, 3, 1, 64), (64, 16, 2, 64)])
def test_cascade(bs, hq, hkv, d):
    pool, ref, table, lens, rng = _filled(bs, hkv, d, [6 * bs + 5, 7 * bs, 5 * bs + 1, bs - 1, 9 * bs], seed=bs)
    table[1:, :5] = table[0, :5]
    q = rng.standard_normal((5, hq, d)).astype(np.float16)
    want = ref.decode(q, table, lens)
    for prefix in range(6):
        out = pool.cascade_decode(_t(q), _t(table), _t(lens), int(lens.max()), prefix)
        assert pool.error() == kvq.KVQ_OK
        _near(out.cpu().numpy(), want)
    pool.close()
