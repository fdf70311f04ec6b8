"""Log-sum-exps, accumulated attention weights and block eviction against float64
definitions, and all of it together as a serving loop runs it."""
import math

import numpy as np
import pytest
import torch

import oracle
import paged_quantized_kv_kvq_gb300 as kvq
from cache_ops_ref import BlockCache, attention, frequencies, rope, tokens
from kvq_testutil import TOL

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
FORMATS = [(kvq.KVQ_FP16, 0), (kvq.KVQ_INT8_PER_TOKEN, 0), (kvq.KVQ_INT8_PER_CHANNEL, 0), (kvq.KVQ_INT8_PER_GROUP, 128),
           (kvq.KVQ_INT8_PER_GROUP, 16), (kvq.KVQ_INT8_PER_GROUP, 32), (kvq.KVQ_FP8_E4M3_PER_TOKEN, 0),
           (kvq.KVQ_INT4_PER_GROUP, 64), (kvq.KVQ_INT4_PER_GROUP, 16), (kvq.KVQ_FP8_E5M2, 0),
           (kvq.KVQ_INT8_PER_BLOCK, 0), (kvq.KVQ_FP8_E4M3_PER_BLOCK, 0)]


def _t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


class Case:
    """A filled pool beside its float64 values."""

    def __init__(self, fmt, group, bs, hq, hkv, d, lens, seed=0, fill_byte=None, spare=3):
        rng = self.rng = np.random.default_rng(seed)
        self.bs, self.hq, self.hkv, self.d = bs, hq, hkv, d
        self.lens = np.array(lens, np.int32)
        per = [(n + bs - 1) // bs for n in lens]
        self.nb = sum(per) + spare
        perm = rng.permutation(self.nb)
        self.table = np.zeros((len(lens), max(max(per), 1) + 2), np.int32)
        at = 0
        for s, p in enumerate(per):
            self.table[s, :p] = perm[at:at + p]
            at += p
        self.spare = perm[at:]
        slots = np.concatenate([tokens(self.table, self.lens, s, bs) for s in range(len(lens))])
        k, v = self.rows(len(slots)), self.rows(len(slots))
        group = min(group, d)
        self.pool = kvq.KVPool(self.nb, bs, hkv, d, fmt, group, device=DEV, fill_byte=fill_byte)
        if fmt in kvq.BLOCK_FORMATS:
            self.ref = BlockCache(fmt, self.nb, bs, hkv, d)
        else:
            self.ref = oracle.OracleCache(fmt, self.nb, bs, hkv, d, group)
        if fmt == kvq.KVQ_INT8_PER_CHANNEL:
            ch = np.full((hkv, d), 0.05, np.float32)
            kvq.kvq_set_channel_scales(self.pool.handle, _t(ch), _t(ch))
            self.ref.set_channel_scales(ch, ch)
        self.pool.append(_t(k), _t(v), _t(slots))
        self.ref.append(k, v, slots)
        self.q = rng.standard_normal((len(lens), hq, d)).astype(np.float16)

    def rows(self, T):
        x = self.rng.standard_normal((T, self.hkv, self.d)).astype(np.float16)
        x[..., ::23] *= 4
        return x

    def values(self, s, table=None, lens=None):
        at = tokens(self.table if table is None else table, self.lens if lens is None else lens, s, self.bs)
        if isinstance(self.ref, BlockCache):
            return self.ref.values(at)
        return np.stack([self.ref.dequantized(kv)[at] for kv in (0, 1)], 1)

    def expect(self, table=None, lens=None):
        return attention(lambda s: self.values(s, table, lens), self.q, self.lens if lens is None else lens)

    def args(self):
        return _t(self.q), _t(self.table), _t(self.lens), int(max(self.lens.max(), 1))


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("bs,hq,hkv,d,lens", [(16, 8, 2, 128, [1, 0, 17, 700, 64]), (32, 5, 1, 64, [33, 400]),
                                              (8, 24, 2, 128, [9, 300, 0]), (64, 4, 4, 64, [65, 129, 1000])])
def test_lse_and_weights(fmt, group, bs, hq, hkv, d, lens):
    if bs == 8 and fmt == kvq.KVQ_INT4_PER_GROUP:
        pytest.skip("INT4 takes blocks of 16 tokens or more")
    c = Case(fmt, group, bs, hq, hkv, d, lens, seed=bs + fmt, fill_byte=0x7F if fmt in (0, 4, 6, 8) else None)
    q, table, L, most = c.args()
    out, lse = c.pool.decode_lse(q, table, L, most)
    assert c.pool.error() == kvq.KVQ_OK
    assert torch.equal(out, c.pool.decode(q, table, L, most))
    want, wl, ww = c.expect()
    np.testing.assert_allclose(out.cpu().numpy(), want, rtol=0, atol=TOL)
    # scores of |z| <= 40 or so within 2^-21 of themselves, the sum of exps within 2^-20
    got = lse.cpu().numpy()
    assert (np.isneginf(got) == np.isneginf(wl)).all()
    np.testing.assert_allclose(got[np.isfinite(wl)], wl[np.isfinite(wl)], rtol=2.0 ** -19, atol=2.0 ** -16)
    for split in (1, 5):
        l2 = torch.empty_like(lse)
        o2 = torch.empty_like(out)
        ws = torch.empty(kvq.kvq_decode_workspace_bytes(c.pool.handle, len(lens), hq, most, split), dtype=torch.uint8, device=DEV)
        kvq.kvq_paged_decode_lse(c.pool.handle, q, table, L, most, d ** -0.5, o2, l2, ws, split)
        np.testing.assert_allclose(l2.cpu().numpy()[np.isfinite(wl)], wl[np.isfinite(wl)], rtol=2.0 ** -19, atol=2.0 ** -16)
    # weights: exp of a difference of two such numbers, relative 2^-14 at worst
    T = most + 5
    prev = np.zeros((len(lens), hkv, T), np.float32)
    for s, n in enumerate(lens):
        prev[s, :, :n] = c.rng.random((hkv, n))
    for p, decay in ((None, 1.0), (prev, 0.75)):
        scores = torch.full((len(lens), hkv, T), -3.0, device=DEV)
        kvq.kvq_attention_weights(c.pool.handle, q, table, L, most, d ** -0.5, lse, scores, None if p is None else _t(p), decay)
        assert c.pool.error() == kvq.KVQ_OK
        got = scores.cpu().numpy()
        for s, n in enumerate(lens):
            assert (got[s, :, n:] == -3.0).all()
            if n:
                w = ww[s].sum(1) + (0 if p is None else decay * p[s, :, :n].astype(np.float64))
                np.testing.assert_allclose(got[s, :, :n], w, rtol=2.0 ** -14, atol=1e-9)
                if p is None:  # every token's weights add up to the heads of the group
                    np.testing.assert_allclose(got[s, :, :n].astype(np.float64).sum(-1), hq // hkv, rtol=2.0 ** -14)
    # in place
    scores = _t(prev)
    c.pool.accumulate_weights(q, table, L, most, lse, scores, 0.75)
    for s, n in enumerate(lens):
        assert np.array_equal(scores.cpu().numpy()[s, :, :n], got[s, :, :n])
    c.pool.close()


def test_weights_skip_bad_blocks_and_empty_rows():
    c = Case(kvq.KVQ_INT8_PER_GROUP, 128, 16, 4, 2, 128, [100, 90], seed=1)
    q, table, L, most = c.args()
    _, lse = c.pool.decode_lse(q, table, L, most)
    ww = c.expect()[2]
    bad = c.table.copy()
    bad[0, 2], bad[1, 5] = -1, c.nb
    lse[1, :2] = -math.inf
    scores = torch.full((2, 2, 112), 5.0, device=DEV)
    kvq.kvq_attention_weights(c.pool.handle, q, _t(bad), L, most, 128 ** -0.5, lse, scores)
    assert c.pool.error() == kvq.KVQ_ERR_OUT_OF_RANGE
    got = scores.cpu().numpy()
    assert (got[0, :, 32:48] == 5).all() and (got[1, :, 80:] == 5).all()
    keep = np.r_[0:32, 48:100]
    np.testing.assert_allclose(got[0][:, keep], ww[0].sum(1)[:, keep], rtol=2.0 ** -14)
    assert (got[1, 0, :80] == 0).all()  # a row that attends nothing weighs nothing
    np.testing.assert_allclose(got[1, 1, :80], ww[1].sum(1)[1, :80], rtol=2.0 ** -14)
    # a length beyond the promised one is clamped and flagged
    scores.fill_(5)
    kvq.kvq_attention_weights(c.pool.handle, q, table, _t(np.array([100, 50], np.int32)), 64, 128 ** -0.5, lse, scores)
    assert c.pool.error() == kvq.KVQ_ERR_OUT_OF_RANGE
    assert (scores.cpu().numpy()[0, :, 64:] == 5).all()
    c.pool.close()


# ------------------------------------------------------------------ eviction
def evict_ref(w, table, lens, bs, budget, sink, recent, width):
    """The definition, one sequence after the other (w fp32; sums in float64)."""
    S, hkv, _ = w.shape
    t2, l2 = table.copy(), lens.copy()
    kept, out = np.full((S, budget), -1, np.int32), {}
    for s in range(S):
        n = -(-int(lens[s]) // bs)
        must = {j for j in range(n) if j < sink or j >= n - recent}
        with np.errstate(invalid="ignore"):
            b = [np.float32(w[s, :, j * bs:min(lens[s], (j + 1) * bs)].astype(np.float64).sum()) for j in range(n)]
        b = [-math.inf if math.isnan(x) else float(x) for x in b]
        free = sorted((j for j in range(n) if j not in must), key=lambda j: (-b[j], j))
        keep = sorted(must | set(free[:max(0, budget - len(must))])) if n > budget else list(range(n))
        gone = [j for j in range(n) if j not in set(keep)]
        t2[s, :n] = table[s, keep + gone]
        kept[s, :len(keep)] = keep
        l2[s] = lens[s] - len(gone) * bs
        at = np.concatenate([np.arange(j * bs, min((j + 1) * bs, lens[s])) for j in keep]).astype(int) if keep else np.zeros(0, int)
        out[s] = w[s][:, at]
    return t2, l2, kept, out


def _evict(pool, w, table, lens, most, budget, sink, recent, extra=3):
    S, hkv, _ = w.shape
    W = budget * pool.block_size + extra
    o = dict(table_out=torch.full(table.shape, -9, dtype=torch.int32, device=DEV), lens_out=torch.empty(S, dtype=torch.int32, device=DEV),
             kept=torch.empty((S, budget), dtype=torch.int32, device=DEV), scores_out=torch.full((S, hkv, W), -7.0, device=DEV))
    kvq.kvq_evict_blocks(pool.handle, _t(w), _t(table), _t(lens), most, budget, sink, recent, **o)
    return {k: v.cpu().numpy() for k, v in o.items()}


def _check_evict(got, want, lens):
    t2, l2, kept, out = want
    np.testing.assert_array_equal(got["table_out"], t2)
    np.testing.assert_array_equal(got["lens_out"], l2)
    np.testing.assert_array_equal(got["kept"], kept)
    for s in range(len(lens)):
        np.testing.assert_array_equal(got["scores_out"][s, :, :l2[s]], out[s])
        assert (got["scores_out"][s, :, l2[s]:] == -7).all()


@pytest.mark.parametrize("bs,hkv,lens,budget,sink,recent", [
    (16, 2, [0, 1, 16, 17, 200, 333], 5, 1, 2), (8, 3, [0, 8, 9, 801, 64], 10, 0, 1), (64, 1, [1000, 64, 65, 3], 3, 0, 1),
    (32, 8, [5000, 4097, 31], 40, 4, 8), (16, 1, [9000], 1, 0, 1), (16, 4, [40000, 12345], 700, 3, 16),
    (8, 2, [30000], 3000, 0, 5), (64, 32, [1500, 900, 2048], 7, 3, 4)])
@pytest.mark.parametrize("kind", ["random", "ties", "wild"])
def test_evict(bs, hkv, lens, budget, sink, recent, kind):
    rng = np.random.default_rng(bs + hkv)
    lens = np.array(lens, np.int32)
    S, most = len(lens), int(lens.max())
    w = rng.random((S, hkv, most + 2)).astype(np.float32) ** 8
    if kind == "ties":
        w = rng.integers(0, 3, w.shape).astype(np.float32) / 4
    if kind == "wild":  # infinities, NaN, negative sums, signed zeros
        w[rng.random(w.shape) < 0.002] = np.nan
        w[rng.random(w.shape) < 0.002] = np.inf
        w[rng.random(w.shape) < 0.3] *= -1
        w[:, :, :most // 3] = -0.0
    for s in range(S):
        w[s, :, lens[s]:] = np.nan  # what lies behind a sequence does not count
    table = rng.permutation(S * (most // bs + 4)).reshape(S, -1).astype(np.int32)
    pool = kvq.KVPool(1, bs, hkv, 64, kvq.KVQ_FP16, device=DEV)
    got = _evict(pool, w, table, lens, most, budget, sink, recent)
    assert pool.error() == kvq.KVQ_OK
    _check_evict(got, evict_ref(w, table, lens, bs, budget, sink, recent, 0), lens)
    pool.close()


def test_evict_sums_do_not_depend_on_their_order():
    """Blocks whose fp32 sums would swap with the order of the additions."""
    rng = np.random.default_rng(0)
    bs, hkv, n = 16, 8, 400
    w = (rng.random((1, hkv, n * bs)) * 10.0 ** rng.integers(-6, 3, (1, hkv, n * bs))).astype(np.float32)
    w[:, :, bs:] = np.tile(w[:, :, :bs], (1, 1, n - 1))
    for j in range(n):  # the same values, shuffled within each block: all sums equal
        w[0, :, j * bs:(j + 1) * bs] = rng.permutation(w[0, :, :bs].ravel()).reshape(hkv, bs)
    # and every third block a little more, by less than fp32 sums would resolve
    for j in range(0, n, 3):
        x = w[0, 0, j * bs:(j + 1) * bs]
        i = int(np.argmax(x))
        x[i] = np.nextafter(x[i], np.float32(np.inf))
    table = np.arange(n, dtype=np.int32)[None]
    lens = np.array([n * bs], np.int32)
    pool = kvq.KVPool(1, bs, hkv, 64, kvq.KVQ_FP16, device=DEV)
    got = _evict(pool, w, table, lens, n * bs, 100, 1, 1)
    _check_evict(got, evict_ref(w, table, lens, bs, 100, 1, 1, 0), lens)
    pool.close()


def test_evict_in_place_and_without_extras():
    rng = np.random.default_rng(4)
    bs, hkv = 16, 2
    lens = np.array([300, 50, 3000], np.int32)
    w = rng.random((3, hkv, 3000)).astype(np.float32)
    table = rng.permutation(600).reshape(3, 200).astype(np.int32)
    pool = kvq.KVPool(1, bs, hkv, 64, kvq.KVQ_FP16, device=DEV)
    t, l = _t(table), _t(lens)
    kvq.kvq_evict_blocks(pool.handle, _t(w), t, l, 3000, 12, 2, 3, t, l)
    t2, l2, _, _ = evict_ref(w, table, lens, bs, 12, 2, 3, 0)
    np.testing.assert_array_equal(t.cpu().numpy(), t2)
    np.testing.assert_array_equal(l.cpu().numpy(), l2)
    # nothing more to do the second time
    kvq.kvq_evict_blocks(pool.handle, _t(w), t, l, 3000, 12, 2, 3, t, l)
    np.testing.assert_array_equal(t.cpu().numpy(), t2)
    # a length beyond the promised one is clamped and flagged
    got = _evict(pool, w, table, np.array([300, 50, 3000], np.int32), 2000, 12, 2, 3)
    assert pool.error() == kvq.KVQ_ERR_OUT_OF_RANGE
    want = evict_ref(w, table, np.array([300, 50, 2000], np.int32), bs, 12, 2, 3, 0)
    _check_evict(got, want, lens)
    pool.close()


def test_evict_of_the_most_blocks():
    """28672 blocks, the largest row; one more is refused."""
    rng = np.random.default_rng(7)
    bs, n = 8, 28672
    w = rng.random((1, 1, n * bs)).astype(np.float32)
    table = rng.permutation(n + 1).astype(np.int32)[None]
    lens = np.array([n * bs - 3], np.int32)
    pool = kvq.KVPool(1, bs, 1, 64, kvq.KVQ_FP16, device=DEV)
    got = _evict(pool, w, table, lens, n * bs, 10000, 4, 64)
    _check_evict(got, evict_ref(w, table, lens, bs, 10000, 4, 64, 0), lens)
    with pytest.raises(kvq.KVQError) as e:
        _evict(pool, np.zeros((1, 1, n * bs + 1), np.float32), table, lens, n * bs + 1, 10000, 4, 64)
    assert e.value.status == kvq.KVQ_ERR_UNSUPPORTED
    pool.close()


@pytest.mark.parametrize("fmt,group", [(kvq.KVQ_INT8_PER_BLOCK, 0), (kvq.KVQ_INT8_PER_GROUP, 64), (kvq.KVQ_FP8_E4M3_PER_BLOCK, 0)])
def test_serving_loop(fmt, group):
    """Prompts come in rotated and normed, then decode steps collect weights, and
    every few steps the sequences are cut to their budget: outputs against a
    float64 attention over what the cache holds."""
    rng = np.random.default_rng(11)
    bs, hq, hkv, d, budget = 16, 8, 2, 64, 6
    lens = np.array([150, 70, 33], np.int32)
    S, W = 3, 256
    pool = kvq.KVPool(64, bs, hkv, d, fmt, group, device=DEV)
    plan = kvq.kvq_rope_init(d, scaling=kvq.KVQ_ROPE_BASE, factor=2.0)
    freq = frequencies(d, scaling=2, factor=2.0)
    weight = _t(1 + 0.2 * rng.standard_normal(d).astype(np.float32))
    table = rng.permutation(64)[:S * 16].reshape(S, 16).astype(np.int32)
    pos = lens.astype(np.int64).copy()

    def feed(at, positions):
        T = len(at)
        qkv = _t(rng.standard_normal((T, hq + 2 * hkv, d)).astype(np.float32)).to(torch.bfloat16)
        q = pool.rope_append(plan, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], _t(positions), _t(at),
                             q_weight=weight, k_weight=weight)
        want = rope(qkv[:, :hq].float().cpu().numpy(), positions, freq, weight=weight.cpu().numpy(), eps=1e-6)
        np.testing.assert_allclose(q.float().cpu().numpy(), want, rtol=2.0 ** -10, atol=2.0 ** -10)
        return q

    feed(np.concatenate([tokens(table, lens, s, bs) for s in range(S)]), np.concatenate([np.arange(n) for n in lens]))
    scores = torch.zeros((S, hkv, W), device=DEV)
    tally = np.zeros((S, hkv, W))
    for step in range(12):
        lens += 1
        at = np.array([tokens(table, lens, s, bs)[-1] for s in range(S)])
        q = feed(at, pos.copy())
        pos += 1
        T, L, most = _t(table), _t(lens), int(lens.max())
        out, lse = pool.decode_lse(q, T, L, most)
        pool.accumulate_weights(q, T, L, most, lse, scores, decay=0.9)
        assert pool.error() == kvq.KVQ_OK

        def values(s):
            k, v = pool.read_values(_t(tokens(table, lens, s, bs)))
            return torch.stack([k, v], 1).double().cpu().numpy()

        want, _, ww = attention(values, q.float().cpu().numpy(), lens)
        # values are read back as fp16: 2^-11 of each
        np.testing.assert_allclose(out.cpu().numpy(), want, rtol=0, atol=4e-3)
        for s in range(S):
            n = lens[s]
            tally[s, :, :n] = 0.9 * tally[s, :, :n] + ww[s].sum(1)
            tally[s, :, n:] = 0
        np.testing.assert_allclose(scores.cpu().numpy(), tally, rtol=0, atol=4e-3)
        if step % 4 == 3:
            w = scores.cpu().numpy()
            t2, l2, kept, outw = evict_ref(w, table, lens, bs, budget, 1, 2, 0)
            nt, nl, nk, ns = pool.evict_blocks(scores, T, L, most, budget, 1, 2)
            np.testing.assert_array_equal(nt.cpu().numpy(), t2)
            np.testing.assert_array_equal(nl.cpu().numpy(), l2)
            np.testing.assert_array_equal(nk.cpu().numpy(), kept)
            new = np.zeros_like(tally)
            for s in range(S):
                np.testing.assert_array_equal(ns.cpu().numpy()[s, :, :l2[s]], outw[s])
                old = np.concatenate([np.arange(j * bs, min((j + 1) * bs, lens[s])) for j in kept[s] if j >= 0])
                new[s][:, :len(old)] = tally[s][:, old]
            table, lens, scores, tally = nt.cpu().numpy(), nl.cpu().numpy(), ns[:, :, :W].contiguous(), new
    assert lens.max() <= budget * bs + 4
    pool.close()


@pytest.mark.parametrize("fmt,group", [(kvq.KVQ_INT8_PER_BLOCK, 0), (kvq.KVQ_INT8_PER_GROUP, 128)])
def test_blocks_beyond_four_gigabytes(fmt, group):
    """Pages whose offsets need more than 32 bits, through every call on them."""
    rng = np.random.default_rng(6)
    nb, bs, hkv, hq, d = 140000, 16, 8, 16, 128  # 4.6 GB
    lens = np.array([700, 1, 90], np.int32)
    small = np.zeros((3, 44), np.int32)
    small[0], small[1, 0], small[2, :6] = np.arange(44), 44, 45 + np.arange(6)
    far = nb - 1 - 37 * rng.permutation(51)
    table = far[small].astype(np.int32)
    ref = BlockCache(fmt, 51, bs, hkv, d) if fmt in kvq.BLOCK_FORMATS else oracle.OracleCache(fmt, 51, bs, hkv, d, group)
    pool = kvq.KVPool(nb, bs, hkv, d, fmt, group, device=DEV)
    near, there = (np.concatenate([tokens(t, lens, s, bs) for s in range(3)]) for t in (small, table))
    k, v = (rng.standard_normal((len(near), hkv, d)).astype(np.float16) for _ in range(2))
    kvq.kvq_rope_append(pool.handle, None, None, _t(k), _t(v), None, _t(there))
    ref.append(k, v, near)
    values = (lambda at: ref.values(at)) if fmt in kvq.BLOCK_FORMATS else \
        (lambda at: np.stack([ref.dequantized(kv)[at] for kv in (0, 1)], 1))
    got = torch.stack(pool.read_values(_t(there)), 1).cpu().numpy()
    np.testing.assert_array_equal(got, values(near).astype(np.float32).astype(np.float16))
    q = rng.standard_normal((3, hq, d)).astype(np.float16)
    out, lse, w = attention(lambda s: values(tokens(small, lens, s, bs)), q, lens)
    o, e = pool.decode_lse(_t(q), _t(table), _t(lens), 700)
    np.testing.assert_allclose(o.cpu().numpy(), out, rtol=0, atol=TOL)
    np.testing.assert_allclose(e.cpu().numpy(), lse, rtol=2.0 ** -19, atol=2.0 ** -16)
    scores = torch.zeros((3, hkv, 704), device=DEV)
    pool.accumulate_weights(_t(q), _t(table), _t(lens), 700, e, scores)
    for s in range(3):
        np.testing.assert_allclose(scores[s, :, :lens[s]].cpu().numpy(), w[s].sum(1), rtol=2.0 ** -14, atol=1e-9)
    assert pool.error() == kvq.KVQ_OK
    pool.close()
