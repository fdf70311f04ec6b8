"""Blocks with one scale each that were filled token by token in memory full of NaN
codes: what lies behind a sequence reaches no result of any way to attend or read."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq
from cache_ops_ref import BlockCache, attention, frequencies, rope, tokens
from kvq_testutil import TOL

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


@pytest.mark.parametrize("fmt", kvq.BLOCK_FORMATS)
@pytest.mark.parametrize("bs,d,lens", [(16, 128, [37, 20, 33]), (8, 64, [19, 17, 30]), (32, 64, [70, 65, 66]), (64, 128, [130, 129, 150])])
def test_blocks_filled_token_by_token(fmt, bs, d, lens):
    rng = np.random.default_rng(bs + fmt)
    hq, hkv, S = 8, 2, 3
    lens = np.array(lens, np.int32)
    per = -(-lens // bs)
    table = np.zeros((S, per.max() + 1), np.int32)
    perm, at = rng.permutation(per.sum() + 3), 0
    for s in range(S):
        table[s, :per[s]] = perm[at:at + per[s]]
        at += per[s]
    table[1:, 0] = table[0, 0]  # one block shared by all
    pool = kvq.KVPool(len(perm), bs, hkv, d, fmt, device=DEV, fill_byte=0x7F)
    ref = BlockCache(fmt, len(perm), bs, hkv, d)
    for t in range(lens.max()):
        who = [s for s in range(S) if t < lens[s] and (s == 0 or t >= bs)]
        slots = np.array([table[s, t // bs] * bs + t % bs for s in who], np.int64)
        k, v = (rng.standard_normal((len(who), hkv, d)).astype(np.float16) * (1 + t % 5) for _ in range(2))
        pool.append(_t(k), _t(v), _t(slots))
        ref.append(k, v, slots)
    q = rng.standard_normal((S, hq, d)).astype(np.float16)
    T, L, most = _t(table), _t(lens), int(lens.max())
    want, wl, ww = attention(lambda s: ref.values(tokens(table, lens, s, bs)), q, lens)
    out, lse = pool.decode_lse(_t(q), T, L, most)
    outs = [out] + ([pool.cascade_decode(_t(q), T, L, most, 1)] if bs >= 16 else [])  # (no cascade over blocks of 8)
    for got in outs:
        np.testing.assert_allclose(got.cpu().numpy(), want, rtol=0, atol=TOL)
    scores = torch.zeros((S, hkv, most), device=DEV)
    pool.accumulate_weights(_t(q), T, L, most, lse, scores)
    for s in range(S):
        np.testing.assert_allclose(scores[s, :, :lens[s]].cpu().numpy(), ww[s].sum(1), rtol=2.0 ** -14, atol=1e-9)
        slots = tokens(table, lens, s, bs)
        got = torch.stack(pool.read_values(_t(slots)), 1).cpu().numpy()
        np.testing.assert_array_equal(got, ref.values(slots).astype(np.float32).astype(np.float16))
    n = [int(x) - bs for x in lens]
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    qq = rng.standard_normal((start[-1], hq, d)).astype(np.float16)
    want = np.concatenate([ref.decode(qq[start[s]:start[s + 1]], np.repeat(table[s:s + 1], n[s], 0),
                                      np.arange(lens[s] - n[s], lens[s]) + 1) for s in range(S)])
    got = torch.empty((int(start[-1]), hq, d), device=DEV)
    ws = torch.empty(kvq.kvq_prefill_workspace_bytes(pool.handle, S, most), dtype=torch.uint8, device=DEV)
    for call, extra in ((kvq.kvq_prefill, ()), (kvq.kvq_prefill_ex, (ws,))) if bs >= 16 else ():  # (nor prefill)
        got.fill_(9)
        call(pool.handle, _t(qq), _t(start), max(n), T, L, most, d ** -0.5, got, *extra)
        np.testing.assert_allclose(got.cpu().numpy(), want, rtol=0, atol=TOL)
    assert pool.error() == kvq.KVQ_OK
    pool.close()


@pytest.mark.parametrize("fmt,group", [(kvq.KVQ_INT8_PER_BLOCK, 0), (kvq.KVQ_FP8_E4M3_PER_BLOCK, 0), (kvq.KVQ_INT8_PER_GROUP, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_keys_of_a_serving_loop(fmt, group, interleaved):
    """A normed and rotated prompt, then steps: the keys read back are the rotated ones
    (not only the same wherever they are read)."""
    rng = np.random.default_rng(3)
    bs, hq, hkv, d, L0, steps = 16, 4, 2, 128, 43, 9
    pool = kvq.KVPool(8, bs, hkv, d, fmt, group, device=DEV)
    plan = kvq.kvq_rope_init(d, interleaved, scaling=kvq.KVQ_ROPE_LINEAR, factor=2.0)
    freq = frequencies(d, scaling=1, factor=2.0)
    w = _t(1 + 0.2 * rng.standard_normal(d).astype(np.float32))
    keys = []
    first = 0
    for n in [L0] + [1] * steps:
        qkv = _t(rng.standard_normal((n, hq + 2 * hkv, d)).astype(np.float32)).to(torch.bfloat16)
        pos = np.arange(first, first + n)
        pool.rope_append(plan, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], _t(pos), _t(pos), q_weight=w, k_weight=w)
        keys.append(rope(qkv[:, hq:hq + hkv].float().cpu().numpy(), pos, freq, interleaved, weight=w.cpu().numpy(), eps=1e-6))
        first += n
    want = np.concatenate(keys)
    got = pool.read_values(torch.arange(first, device=DEV))[0].double().cpu().numpy()
    # a code's half step (of the block's, or group's, largest key), once more for each
    # time that its block's scale grew: at most once a token behind it
    top = 448.0 if fmt == kvq.KVQ_FP8_E4M3_PER_BLOCK else 127.0
    for b in range(-(-first // bs)):
        at = slice(b * bs, min((b + 1) * bs, first))
        a = np.abs(want[at]).max((0, 2), keepdims=True)
        half = np.abs(want[at]) * 2.0 ** -4 + a / top * 2.0 ** -10 if top == 448.0 else np.broadcast_to(a / top / 2, want[at].shape)
        grown = 1 + max(0, min((b + 1) * bs, first) - max(b * bs, L0)) if fmt in kvq.BLOCK_FORMATS else 1
        assert (np.abs(got[at] - want[at]) <= half * (1.07 ** grown) * grown + 2.0 ** -10 * np.abs(want[at]) + 2.0 ** -16).all()
    assert pool.error() == kvq.KVQ_OK
    pool.close()
