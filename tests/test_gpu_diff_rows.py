"""Differential prompts write the rows of the sequences and no others, in every format."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq
from cache_ops_ref import tokens
from test_gpu_diff import DEV, FORMATS, SUMS, _filled, _near, _t, diff_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_rows_around_the_sequences_stay(fmt, group):
    """Rows before q_start[0], which another call may hold, and behind the last sequence; the
    workspace is filled with NaN."""
    bs, H, hkv, d = 16, 4, 2, 128
    pool, vals, table, lens, rng = _filled(fmt, group, bs, hkv, d, [40, 0, 90], seed=4)
    n, first, T = [40, 0, 30], 5, 81
    start = (first + np.concatenate([[0], np.cumsum(n)])).astype(np.int32)
    end = int(start[-1])
    q = rng.standard_normal((T, H, d)).astype(np.float16)
    lam, w = rng.uniform(-0.5, 1, H).astype(np.float32), rng.uniform(0.5, 1.5, d).astype(np.float32)
    rows_lens = np.concatenate([np.arange(lens[s] - n[s], lens[s]) + 1 for s in range(3)]).astype(np.int32)
    seq = np.repeat(np.arange(3), n)
    want, maps = diff_ref(lambda r: vals[tokens(table[seq], rows_lens, r, bs)], q[first:end], rows_lens, lam.astype(np.float64), w, 1e-5, 0.2)
    ws = torch.full((kvq.kvq_diff_prefill_workspace_bytes(pool.handle, 3, T, H, 90),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full((T, H, d), 7.0, dtype=torch.float16, device=DEV)
    kvq.kvq_diff_prefill(pool.handle, _t(q), _t(start), 40, _t(table), _t(lens), 90, (d // 2) ** -0.5, _t(lam), out, ws, _t(w), 1e-5, 0.2)
    assert pool.error() == kvq.KVQ_OK
    assert (out[:first] == 7).all() and (out[end:] == 7).all()
    _near(out[first:end].cpu().numpy(), want, maps, lam, w, 0.2, SUMS)
    pool.close()
