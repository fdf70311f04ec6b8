"""Pools with one scale per (block, kv head): codes and scales bit by bit against
the format's definition through every way to append, attention against float64
through every way to attend."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq
from cache_ops_ref import BlockCache, attention, tokens
from kvq_testutil import TOL

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
FORMATS = [kvq.KVQ_INT8_PER_BLOCK, kvq.KVQ_FP8_E4M3_PER_BLOCK]
# Attention outputs: scores carry |z| <= ~16 within 2^-21 of themselves (fp32 sums
# of exact products), so weights are within 1e-5 of themselves; P.V adds 2^-22.
REL = 1e-5


def _t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _rows(rng, T, hkv, d):
    x = rng.standard_normal((T, hkv, d)).astype(np.float16)
    x[:, :, ::29] *= 8
    x[rng.random(T) < 0.1] *= 5  # tokens that make a block's scale grow
    return x


def _check(pool, ref, slots):
    codes, scales = pool.read_slots(_t(slots))
    np.testing.assert_array_equal(codes.cpu().numpy().view(np.uint8), ref.codes[slots].view(np.uint8))
    np.testing.assert_array_equal(scales.cpu().numpy().view(np.uint32),
                                  ref.scales[slots // ref.bs].view(np.uint32))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bs,hkv,d", [(16, 2, 128), (8, 3, 64), (32, 1, 64), (64, 2, 128), (8, 1, 128),
                                      (16, 5, 64), (32, 2, 128), (64, 1, 64), (16, 11, 128), (32, 33, 64)])
def test_append_is_bit_exact(fmt, bs, hkv, d):
    """Prompts (whole, ragged, starting inside a block), single tokens that grow or
    keep a scale, padding, a block begun anew."""
    rng = np.random.default_rng(fmt * 1000 + bs + hkv)
    nb = 24
    pool = kvq.KVPool(nb, bs, hkv, d, fmt, device=DEV)
    ref = BlockCache(fmt, nb, bs, hkv, d)
    perm = rng.permutation(nb)

    def put(slots):
        slots = np.asarray(slots, np.int64)
        k, v = _rows(rng, len(slots), hkv, d), _rows(rng, len(slots), hkv, d)
        pool.append(_t(k), _t(v), _t(slots))
        ref.append(k, v, slots)

    def seq(first, t0, n):  # n tokens from position t0 of the sequence whose blocks start at `first`
        t = np.arange(t0, t0 + n)
        return perm[first + t // bs] * bs + t % bs

    put(seq(0, 0, 3 * bs))                          # whole blocks
    put(np.concatenate([seq(4, 0, bs + 5), seq(8, 0, 1), seq(10, 0, 2 * bs - 1)]))  # ragged
    put(np.concatenate([seq(4, bs + 5, bs), [-1, -1], seq(10, 2 * bs - 1, 3)]))     # go on inside a block
    for i in range(4):                              # decode steps
        put(np.concatenate([seq(8, 1 + i, 1), seq(4, 2 * bs + 5 + i, 1), [-1], seq(0, 3 * bs + i, 1)]))
    put(seq(0, 0, 2))                               # block begun anew: older codes are gone
    used = np.unique(np.concatenate([seq(0, 0, 3 * bs + 4), seq(4, 0, 2 * bs + 9), seq(8, 0, 5),
                                     seq(10, 0, 2 * bs + 2)]))
    assert pool.error() == kvq.KVQ_OK
    _check(pool, ref, used)
    pool.close()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bs,T", [(16, 5000), (64, 3001), (8, 1100)])
def test_append_of_many_tokens(fmt, bs, T):
    """Calls large enough that a CTA takes a block's worth of tokens: sequences that
    end anywhere, runs that start inside a CTA's share and end in the next one's."""
    rng = np.random.default_rng(T)
    hkv, d = 2, 128
    lens = []
    while sum(lens) < T:
        lens.append(int(min(rng.integers(1, 6 * bs), T - sum(lens))))
    per = [(n + bs - 1) // bs for n in lens]
    perm = rng.permutation(sum(per))
    slots, first = [], 0
    for n, p in zip(lens, per):
        t = np.arange(n)
        slots.append(perm[first + t // bs] * bs + t % bs)
        first += p
    slots = np.concatenate(slots)
    k, v = _rows(rng, T, hkv, d), _rows(rng, T, hkv, d)
    pool = kvq.KVPool(first, bs, hkv, d, fmt, device=DEV)
    ref = BlockCache(fmt, first, bs, hkv, d)
    pool.append(_t(k), _t(v), _t(slots))
    ref.append(k, v, slots)
    assert pool.error() == kvq.KVQ_OK
    _check(pool, ref, slots)
    # a strided append of the same rows gives the same blocks
    wide = np.concatenate([k, v], 1)
    pool2 = kvq.KVPool(first, bs, hkv, d, fmt, device=DEV)
    w = _t(wide)
    kvq.kvq_append_strided(pool2.handle, w[:, :hkv], w[:, hkv:], _t(slots))
    _check(pool2, ref, slots)
    pool.close()
    pool2.close()


@pytest.mark.parametrize("fmt,group", [(FORMATS[0], 0), (FORMATS[1], 0), (kvq.KVQ_INT8_PER_GROUP, 32)])
def test_codes_at_the_borders(fmt, group):
    """Whole blocks of values that sit on and next to the codes' borders, zero blocks,
    subnormal and huge scales, infinities and NaN: the bits of the definition (for
    the per-group format, of the append that was there)."""
    rng = np.random.default_rng(12)
    nb, hkv, d, bs = 80, 1, 128, 16
    T = nb * bs
    x = (rng.integers(-127, 128, (T, hkv, d)) + rng.choice([0, 0.5, -0.5, 0.4999, 0.5001], (T, hkv, d))).astype(np.float32)
    scale = 2.0 ** rng.integers(-20, 8, (nb, 1, 1, 1))  # absmax 127 * 2^n: exact ties
    scale[::3] *= rng.random((len(scale[::3]), 1, 1, 1)) + 0.5
    x = (np.clip(x, -127, 127).reshape(nb, bs, hkv, d) * scale)
    x[:, 0, :, ::32] = 127 * scale[:, 0]
    x[5] = 0
    x[6] = 6e-8 * rng.integers(-3, 4, x[6].shape)
    x[7] *= 0
    x[7, 3, 0, 9] = 65504
    x = x.reshape(T, hkv, d).astype(np.float16)
    x[:, 0, 1] = np.minimum(x[:, 0, 1], 60000)
    slots = np.arange(T, dtype=np.int64)
    pool = kvq.KVPool(nb, bs, hkv, d, fmt, group, device=DEV)
    assert pool.rope_append(None, None, _t(x), _t(-x), None, _t(slots)) is None
    codes, scales = pool.read_slots(_t(slots))
    if group:
        other = kvq.KVPool(nb, bs, hkv, d, fmt, group, device=DEV)
        other.append(_t(x), _t(-x), _t(slots))
        c2, s2 = other.read_slots(_t(slots))
        assert torch.equal(codes, c2) and torch.equal(scales, s2)
        x[100:130, 0, 5] = np.nan
        x[200, 0, 7] = np.inf
        pool.rope_append(None, None, _t(x), _t(-x), None, _t(slots))
        other.append(_t(x), _t(-x), _t(slots))
        for a, b in zip(pool.read_slots(_t(slots)), other.read_slots(_t(slots))):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        other.close()
    else:
        ref = BlockCache(fmt, nb, bs, hkv, d)
        ref.append(x, -x, slots)
        _check(pool, ref, slots)
    pool.close()


@pytest.mark.parametrize("fmt", FORMATS)
def test_out_of_range_slots_are_flagged_and_skipped(fmt):
    rng = np.random.default_rng(3)
    pool = kvq.KVPool(4, 16, 2, 64, fmt, device=DEV)
    ref = BlockCache(fmt, 4, 16, 2, 64)
    slots = np.array([0, 1, 64, 17, 2 ** 40, 16, 63], np.int64)
    k, v = _rows(rng, 7, 2, 64), _rows(rng, 7, 2, 64)
    pool.append(_t(k), _t(v), _t(slots))
    ok = slots < 64
    ref.append(k[ok], v[ok], slots[ok][[0, 1, 2, 3, 4]])
    assert pool.error() == kvq.KVQ_ERR_OUT_OF_RANGE
    _check(pool, ref, np.array([0, 1, 63], np.int64))
    pool.close()


def _filled(fmt, bs, hkv, d, lens, seed=0, fill_byte=None, spare=2):
    rng = np.random.default_rng(seed)
    per = [(n + bs - 1) // bs for n in lens]
    nb = sum(per) + spare
    perm = rng.permutation(nb)
    table = np.zeros((len(lens), max(max(per), 1) + 1), np.int32)
    at = 0
    slots = []
    for s, (n, p) in enumerate(zip(lens, per)):
        table[s, :p] = perm[at:at + p]
        at += p
        t = np.arange(n)
        slots.append(table[s, t // bs].astype(np.int64) * bs + t % bs)
    slots = np.concatenate(slots)
    k, v = _rows(rng, len(slots), hkv, d), _rows(rng, len(slots), hkv, d)
    pool = kvq.KVPool(nb, bs, hkv, d, fmt, device=DEV, fill_byte=fill_byte)
    ref = BlockCache(fmt, nb, bs, hkv, d)
    pool.append(_t(k), _t(v), _t(slots))
    ref.append(k, v, slots)
    return pool, ref, table, np.array(lens, np.int32), rng


def _near(got, want):
    assert np.isfinite(got).all()
    assert np.linalg.norm(got - want) <= REL * np.linalg.norm(want)
    np.testing.assert_allclose(got, want, rtol=0, atol=TOL)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bs,hq,hkv,d,lens", [
    (16, 8, 2, 128, [1, 0, 17, 333, 16, 900]), (8, 8, 2, 128, [1, 0, 7, 8, 9, 301, 64]),
    (32, 4, 1, 64, [31, 33, 500]), (64, 6, 2, 64, [63, 65, 1, 700]), (64, 4, 4, 128, [129, 0, 640]),
    (16, 24, 2, 128, [45, 400]), (16, 32, 1, 64, [250]), (8, 4, 1, 64, [100, 33]),
    (32, 3, 3, 128, [200, 64])])
def test_decode(fmt, bs, hq, hkv, d, lens):
    # 0x7F bytes are NaN as e4m3: what lies behind a sequence must not reach it
    pool, ref, table, lens, rng = _filled(fmt, bs, hkv, d, lens, seed=bs + hq, fill_byte=0x7F)
    q = rng.standard_normal((len(lens), hq, d)).astype(np.float16)
    want = ref.decode(q, table, lens)
    for split in (0, 1, 3):
        out = pool.decode(_t(q), _t(table), _t(lens), int(max(lens.max(), 1)), split_blocks=split)
        assert pool.error() == kvq.KVQ_OK
        _near(out.cpu().numpy(), want)
    wide_q = torch.zeros((len(lens), hq + 3, d), dtype=torch.float16, device=DEV)
    wide_q[:, 2:2 + hq] = _t(q)
    wide = torch.full((len(lens), hq + 1, d), 9.0, device=DEV)
    ws = torch.empty(kvq.kvq_decode_workspace_bytes(pool.handle, len(lens), hq, int(lens.max())), dtype=torch.uint8, device=DEV)
    kvq.kvq_paged_decode_strided(pool.handle, wide_q[:, 2:2 + hq], _t(table), _t(lens), int(lens.max()), d ** -0.5, wide[:, 1:], ws)
    _near(wide[:, 1:].cpu().numpy(), want)
    assert (wide[:, 0] == 9).all()
    out = torch.empty((len(lens), hq, d), device=DEV)
    kvq.kvq_paged_decode_noalloc(pool.handle, _t(q), _t(table), _t(lens), int(lens.max()), d ** -0.5, out)
    _near(out.cpu().numpy(), want)
    pool.close()


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_range_in_one_warp_does_not_drift(fmt):
    """24000 tokens summed by one warp: the sum stays in fp32 adds."""
    pool, ref, table, lens, rng = _filled(fmt, 16, 1, 128, [24000], seed=5)
    q = rng.standard_normal((1, 4, 128)).astype(np.float16)
    want = ref.decode(q, table, lens)
    out = pool.decode(_t(q), _t(table), _t(lens), 24000, split_blocks=1500)
    _near(out.cpu().numpy(), want)
    pool.close()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bs", [8, 16, 64])
def test_decode_steps(fmt, bs):
    """Steps that fill a block, start the next and grow its scale."""
    hq, hkv, d = 8, 2, 128
    pool, ref, table, lens, rng = _filled(fmt, bs, hkv, d, [bs - 2, 5 * bs - 1, 3], seed=1, spare=8)
    spare = np.setdiff1d(np.arange(len(ref.scales)), table.ravel())
    lens = lens.copy()
    for s in range(3):
        n = (lens[s] + bs - 1) // bs
        table[s, n] = spare[s]
    for _ in range(4):
        lens += 1
        k, v = _rows(rng, 3, hkv, d), _rows(rng, 3, hkv, d)
        q = rng.standard_normal((3, hq, d)).astype(np.float16)
        at = np.array([tokens(table, lens, s, bs)[-1] for s in range(3)])
        out = pool.decode_step(_t(k), _t(v), _t(q), _t(table), _t(lens), int(lens.max()))
        ref.append(k, v, at)
        assert pool.error() == kvq.KVQ_OK
        _near(out.cpu().numpy(), ref.decode(q, table, lens))
    _check(pool, ref, np.concatenate([tokens(table, lens, s, bs) for s in range(3)]))
    # a sequence without tokens stores nothing, a bad block is flagged
    k, v = _rows(rng, 3, hkv, d), _rows(rng, 3, hkv, d)
    bad = table.copy()
    bad[1, 0] = -1
    before = pool.buffer[256:].clone()
    pool.decode_step(_t(k), _t(v), _t(q), _t(bad), _t(np.array([0, 1, 0], np.int32)), bs)
    assert pool.error() == kvq.KVQ_ERR_OUT_OF_RANGE
    assert torch.equal(before, pool.buffer[256:])
    pool.close()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bs", [16, 64])
def test_cascade_prefill_and_copies(fmt, bs):
    hq, hkv, d = 8, 2, 128
    pool, ref, table, lens, rng = _filled(fmt, bs, hkv, d, [3 * bs + 5, 4 * bs, 2 * bs], seed=2, spare=9)
    table[1:, :2] = table[0, :2]  # a shared prefix of two blocks
    q = rng.standard_normal((3, hq, d)).astype(np.float16)
    out = pool.cascade_decode(_t(q), _t(table), _t(lens), int(lens.max()), 2)
    np.testing.assert_allclose(out.cpu().numpy(), ref.decode(q, table, lens), rtol=0, atol=TOL)
    # copies of the shared blocks give the same bits
    spare = np.setdiff1d(np.arange(len(ref.scales)), table.ravel())[:2].astype(np.int32)
    kvq.kvq_copy_blocks(pool.handle, _t(table[1, :2]), _t(spare))
    own = table.copy()
    own[1, :2] = spare
    a = pool.decode(_t(q), _t(table), _t(lens), int(lens.max()))
    b = pool.decode(_t(q), _t(own), _t(lens), int(lens.max()))
    assert torch.equal(a, b)
    # prefill: the last n tokens of each sequence attend causally, both entry points
    n = [bs + 3, 1, 2 * bs]
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    qq = rng.standard_normal((start[-1], hq, d)).astype(np.float16)
    want = np.zeros((start[-1], hq, d))
    for s in range(3):
        for i in range(n[s]):
            one = np.array([lens[s] - n[s] + i + 1])
            want[start[s] + i] = ref.decode(qq[start[s] + i][None], table[s:s + 1], one)[0]
    got = torch.empty((start[-1], hq, d), device=DEV)
    kvq.kvq_prefill(pool.handle, _t(qq), _t(start), max(n), _t(table), _t(lens), int(lens.max()), d ** -0.5, got)
    np.testing.assert_allclose(got.cpu().numpy(), want, rtol=0, atol=TOL)
    ws = torch.empty(kvq.kvq_prefill_workspace_bytes(pool.handle, 3, int(lens.max())), dtype=torch.uint8, device=DEV)
    got.zero_()
    kvq.kvq_prefill_ex(pool.handle, _t(qq), _t(start), max(n), _t(table), _t(lens), int(lens.max()), d ** -0.5, got, ws)
    np.testing.assert_allclose(got.cpu().numpy(), want, rtol=0, atol=TOL)
    assert pool.error() == kvq.KVQ_OK
    pool.close()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d,hkv", [(128, 3), (64, 18)])
def test_a_step_of_many_sequences(fmt, d, hkv):
    """1300 sequences, a token each, into blocks that hold tokens already: the form
    that takes several runs per CTA."""
    rng = np.random.default_rng(17)
    bs, S = 16, 1300
    pool = kvq.KVPool(S, bs, hkv, d, fmt, device=DEV)
    ref = BlockCache(fmt, S, bs, hkv, d)
    perm = rng.permutation(S)
    have = rng.integers(0, bs, S)
    for t in range(bs):
        at = perm[have > t] * bs + t
        if t < 3 and len(at):  # (three tokens are enough of a past)
            k, v = _rows(rng, len(at), hkv, d), _rows(rng, len(at), hkv, d)
            pool.append(_t(k), _t(v), _t(at))
            ref.append(k, v, at)
    at = perm * bs + np.minimum(have, 3)
    at[::41] = -1
    k, v = _rows(rng, S, hkv, d), _rows(rng, S, hkv, d)
    pool.append(_t(k), _t(v), _t(at))
    ref.append(k, v, at)
    assert pool.error() == kvq.KVQ_OK
    whole = np.concatenate([perm[i] * bs + np.arange(min(have[i], 3) + 1) for i in range(0, S, 7) if at[i] >= 0])
    _check(pool, ref, whole)
    pool.close()


def test_append_and_step_captured_in_a_graph():
    """A captured append + step replays on what the buffers hold then."""
    fmt, bs, hq, hkv, d = kvq.KVQ_INT8_PER_BLOCK, 16, 4, 1, 64
    pool, ref, table, lens, rng = _filled(fmt, bs, hkv, d, [20, 40], seed=4)
    kb, vb = torch.empty((2, hkv, d), dtype=torch.float16, device=DEV), torch.empty((2, hkv, d), dtype=torch.float16, device=DEV)
    q, L = _t(rng.standard_normal((2, hq, d)).astype(np.float16)), _t(lens)
    tb, out = _t(table), torch.empty((2, hq, d), device=DEV)
    ws = torch.empty(kvq.kvq_decode_workspace_bytes(pool.handle, 2, hq, 48), dtype=torch.uint8, device=DEV)
    kvq.kvq_paged_decode(pool.handle, q, tb, L, 48, d ** -0.5, out, ws)  # warm-up
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        kvq.kvq_decode_step(pool.handle, kb, vb, q, tb, L, 48, d ** -0.5, out, ws)
    for _ in range(3):
        lens += 1
        L.copy_(_t(lens))
        k, v = _rows(rng, 2, hkv, d), _rows(rng, 2, hkv, d)
        kb.copy_(_t(k))
        vb.copy_(_t(v))
        g.replay()
        torch.cuda.synchronize()
        ref.append(k, v, [tokens(table, lens, s, bs)[-1] for s in range(2)])
        _near(out.cpu().numpy(), ref.decode(q.cpu().numpy(), table, lens))
    pool.close()


@pytest.mark.parametrize("fmt,group", [(f, 0) for f in FORMATS] + [
    (kvq.KVQ_FP16, 0), (kvq.KVQ_INT8_PER_TOKEN, 0), (kvq.KVQ_INT8_PER_GROUP, 32), (kvq.KVQ_FP8_E4M3_PER_TOKEN, 0),
    (kvq.KVQ_INT4_PER_GROUP, 64), (kvq.KVQ_FP8_E5M2, 0), (kvq.KVQ_INT8_PER_CHANNEL, 0)])
@pytest.mark.parametrize("bs,d", [(16, 64), (64, 128), (8, 128)])
def test_read_values(fmt, group, bs, d):
    """Values are code * scale rounded to fp16; padding keeps its rows, bad slots are flagged."""
    if bs == 8 and fmt == kvq.KVQ_INT4_PER_GROUP:
        pytest.skip("INT4 takes blocks of 16 tokens or more")
    rng = np.random.default_rng(9)
    nb, hkv = 5, 3
    pool = kvq.KVPool(nb, bs, hkv, d, fmt, group, device=DEV)
    if fmt == kvq.KVQ_INT8_PER_CHANNEL:
        c = _t(_rows(rng, 30, hkv, d))
        kvq.kvq_calibrate_channel_scales(pool.handle, c, c)
        chan = (c.float().abs().amax(0) / torch.full((), 127.0, device=DEV)).cpu().numpy()
    slots = np.arange(nb * bs)
    pool.append(_t(_rows(rng, len(slots), hkv, d)), _t(_rows(rng, len(slots), hkv, d)), _t(slots))
    ask = np.concatenate([rng.permutation(slots)[:37], [-1, 0]])
    k = torch.full((len(ask), hkv, d), 7.0, dtype=torch.float16, device=DEV)
    v = k.clone()
    kvq.kvq_read_values(pool.handle, _t(ask), k, v)
    assert pool.error() == kvq.KVQ_OK
    real = ask >= 0
    codes, scales = pool.read_slots(_t(ask[real]))
    if codes.dtype == torch.uint8:
        codes = codes.view(torch.float8_e5m2 if fmt == kvq.KVQ_FP8_E5M2 else torch.float8_e4m3fn)
    x = codes.float().cpu().numpy()
    if scales is not None:
        s = scales.cpu().numpy()
        s = s[..., None] if fmt in FORMATS else s[..., None, None] if s.ndim == 2 else np.repeat(s, group, -1)
        x = x * s
    elif fmt == kvq.KVQ_INT8_PER_CHANNEL:
        x = x * chan
    for got, want in ((k, x[:, 0]), (v, x[:, 1])):
        got = got.cpu().numpy()
        np.testing.assert_array_equal(got[real], want.astype(np.float16))
        assert (got[~real] == 7.0).all()
    kvq.kvq_read_values(pool.handle, _t(np.array([nb * bs, 1])), k[:2].contiguous(), v[:2].contiguous())
    assert pool.error() == kvq.KVQ_ERR_OUT_OF_RANGE
    pool.close()
