"""NaN scores show in the log-sum-exps and in the weights made from them; a row
without them is untouched by its neighbours'."""
import math

import numpy as np
import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BS, HQ, HKV, D = 16, 8, 2, 128


def _pool(lens, bad=None):
    """FP16 pool of sequences in order; key `bad` = (sequence, token, kv head) is NaN."""
    g = torch.Generator(device=DEV).manual_seed(3)
    per = [-(-n // BS) for n in lens]
    table = torch.zeros((len(lens), max(per)), dtype=torch.int32, device=DEV)
    pool = kvq.KVPool(sum(per), BS, HKV, D, kvq.KVQ_FP16, device=DEV)
    first = 0
    for s, (n, p) in enumerate(zip(lens, per)):
        table[s, :p] = torch.arange(first, first + p)
        k = torch.randn((n, HKV, D), generator=g, device=DEV).half()
        v = torch.randn((n, HKV, D), generator=g, device=DEV).half()
        if bad is not None and bad[0] == s:
            k[bad[1], bad[2], 5] = math.nan
        pool.append(k, v, first * BS + torch.arange(n, device=DEV))
        first += p
    q = torch.randn((len(lens), HQ, D), generator=g, device=DEV).half()
    return pool, q, table, torch.tensor(lens, dtype=torch.int32, device=DEV)


def _lse(pool, q, table, lens, split):
    S, most = len(lens), int(lens.max())
    out, lse = torch.empty((S, HQ, D), device=DEV), torch.empty((S, HQ), device=DEV)
    ws = torch.empty(kvq.kvq_decode_workspace_bytes(pool.handle, S, HQ, most, split), dtype=torch.uint8, device=DEV)
    kvq.kvq_paged_decode_lse(pool.handle, q, table, lens, most, D ** -0.5, out, lse, ws, split)
    assert pool.error() == kvq.KVQ_OK
    return lse


@pytest.mark.parametrize("split", [0, 1, 3, 100])
@pytest.mark.parametrize("token", [0, 17, 699])
def test_a_nan_key(split, token):
    lens = [700, 40, 0]
    clean = _lse(*_pool(lens), split)
    pool, q, table, L = _pool(lens, (0, token, 1))
    lse = _lse(pool, q, table, L, split)
    assert torch.isnan(lse[0, 4:]).all()
    assert torch.equal(lse[0, :4], clean[0, :4]) and torch.equal(lse[1:], clean[1:])
    assert torch.isneginf(lse[2]).all()
    scores = torch.zeros((3, HKV, 704), device=DEV)
    pool.accumulate_weights(q, table, L, 700, lse, scores)
    assert torch.isnan(scores[0, 1, :700]).all() and torch.isfinite(scores[0, 0]).all() and torch.isfinite(scores[1]).all()
    np.testing.assert_allclose(scores[1].sum(-1).cpu().numpy(), HQ // HKV, rtol=2.0 ** -14)


@pytest.mark.parametrize("split", [0, 1, 3, 100])
@pytest.mark.parametrize("lens", [[700, 40], [9, 40]])
def test_a_nan_query(split, lens):
    """Every score of the row is NaN: no maximum is ever found."""
    pool, q, table, L = _pool(lens)
    clean = _lse(pool, q, table, L, split)
    q[0, 2, 9] = math.nan
    lse = _lse(pool, q, table, L, split)
    assert torch.isnan(lse[0, 2])
    lse[0, 2] = clean[0, 2]
    assert torch.equal(lse, clean)
