"""The cache in 4-bit floats: codes and scales bit by bit against the format's definition
through every way to append, attention against float64 through every way to attend."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq
from cache_ops_ref import attention, frequencies, rope, tokens
from fp4_ref import SCALES, Fp4Cache, quantize, values
from kvq_testutil import TOL

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
FMT = kvq.KVQ_FP4_E2M1
# Attention outputs: dequantized values are exact in fp16; scores carry |z| <= ~16 within
# 2^-21 of themselves (fp32 sums of exact products), so weights are within 1e-5 of
# themselves at worst and errors average out; weights enter P.V within 2^-22.
REL = 1e-5


def _t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _rows(rng, T, hkv, d):
    x = rng.standard_normal((T, hkv, d)).astype(np.float16)
    x[:, :, ::29] *= 8
    x[rng.random(T) < 0.1] *= 5
    return x


def _check(pool, ref, slots):
    codes, scales = pool.read_slots(_t(slots))
    np.testing.assert_array_equal(codes.cpu().numpy(), ref.codes[slots])
    np.testing.assert_array_equal(scales.cpu().numpy(), SCALES[ref.scales[slots]].astype(np.float32))
    k, v = pool.read_values(_t(slots))
    want = ref.values(slots)
    np.testing.assert_array_equal(k.cpu().numpy(), want[:, 0].astype(np.float16))
    np.testing.assert_array_equal(v.cpu().numpy(), want[:, 1].astype(np.float16))


def _filled(bs, hkv, d, lens, seed=0, fill_byte=0xFF, spare=0):
    """A pool in memory of `fill_byte` (0xFF: scales that are NaN) with sequences of the given lengths."""
    rng = np.random.default_rng(seed)
    per = [(n + bs - 1) // bs for n in lens]
    nb = max(sum(per), 1) + spare
    perm = rng.permutation(nb)
    table = np.zeros((len(lens), max(max(per), 1) + 2), np.int32)
    slots, at = [], 0
    for s, n in enumerate(lens):
        table[s, :per[s]] = perm[at:at + per[s]]
        at += per[s]
        t = np.arange(n)
        slots.append(table[s, t // bs].astype(np.int64) * bs + t % bs)
    slots = np.concatenate(slots)
    k, v = _rows(rng, len(slots), hkv, d), _rows(rng, len(slots), hkv, d)
    pool = kvq.KVPool(nb, bs, hkv, d, FMT, device=DEV, fill_byte=fill_byte)
    ref = Fp4Cache(nb, bs, hkv, d)
    if len(slots):
        pool.append(_t(k), _t(v), _t(slots))
        ref.append(k, v, slots)
    return pool, ref, table, np.array(lens, np.int32), rng


def _near(got, want):
    assert np.isfinite(got).all()
    assert np.linalg.norm(got - want) <= REL * np.linalg.norm(want)
    np.testing.assert_allclose(got, want, rtol=0, atol=TOL)


# ------------------------------------------------------------------ appends
@pytest.mark.parametrize("way", ["append", "strided", "fused", "fused_bf16"])
@pytest.mark.parametrize("bs,hkv,d", [(16, 2, 128), (32, 1, 64), (64, 2, 128), (16, 5, 64), (16, 11, 128), (32, 33, 64)])
def test_append_is_bit_exact(way, bs, hkv, d):
    """Prompts (whole, ragged, starting inside a block), single tokens, padding, blocks
    begun anew; neighbours of what a call writes stay."""
    rng = np.random.default_rng(1000 + bs + hkv)
    nb = 24
    pool = kvq.KVPool(nb, bs, hkv, d, FMT, device=DEV)
    ref = Fp4Cache(nb, bs, hkv, d)
    perm = rng.permutation(nb)

    def put(slots):
        slots = np.asarray(slots, np.int64)
        k, v = _rows(rng, len(slots), hkv, d), _rows(rng, len(slots), hkv, d)
        if way == "append":
            pool.append(_t(k), _t(v), _t(slots))
        elif way == "strided":
            wide = _t(np.concatenate([k, v], 1))
            kvq.kvq_append_strided(pool.handle, wide[:, :hkv], wide[:, hkv:], _t(slots))
        elif way == "fused":
            pool.rope_append(None, None, _t(k), _t(v), None, _t(slots))
        else:
            kb, vb = _t(k).bfloat16(), _t(v).bfloat16()
            pool.rope_append(None, None, kb, vb, None, _t(slots))
            k, v = kb.float().cpu().numpy(), vb.float().cpu().numpy()
        ref.append(k, v, slots)

    def seq(first, t0, n):
        t = np.arange(t0, t0 + n)
        return perm[first + t // bs] * bs + t % bs

    put(seq(0, 0, 3 * bs))
    put(np.concatenate([seq(4, 0, bs + 5), seq(8, 0, 1), seq(10, 0, 2 * bs - 1)]))
    put(np.concatenate([seq(4, bs + 5, bs), [-1, -1], seq(10, 2 * bs - 1, 3)]))
    for i in range(4):
        put(np.concatenate([seq(8, 1 + i, 1), seq(4, 2 * bs + 5 + i, 1), [-1], seq(0, 3 * bs + i, 1)]))
    put(seq(0, 0, 2))
    put(seq(0, 5, 7)[::-1])  # an order of its own
    used = np.unique(np.concatenate([seq(0, 0, 3 * bs + 4), seq(4, 0, 2 * bs + 9), seq(8, 0, 5), seq(10, 0, 2 * bs + 2)]))
    assert pool.error() == kvq.KVQ_OK
    _check(pool, ref, used)
    pool.close()


@pytest.mark.parametrize("way", ["append", "strided", "fused"])
@pytest.mark.parametrize("bs,hkv,d,T", [(16, 2, 128, 5000), (64, 3, 64, 3001), (32, 1, 128, 1100), (16, 1, 64, 1025), (16, 9, 64, 511),
                                        (16, 3, 128, 512), (32, 5, 64, 2049)])
def test_append_of_many_tokens(way, bs, hkv, d, T):
    """Long calls: sequences that begin and end anywhere in their blocks, whose older
    tokens stay, single tokens and padding among them."""
    rng = np.random.default_rng(T)
    lens = []
    while sum(lens) < T:
        lens.append(int(min(rng.choice([1, 2, rng.integers(1, 6 * bs)]), T - sum(lens))))
    starts = rng.integers(0, bs, len(lens)) * (rng.random(len(lens)) < 0.6)
    per = [(a + n + bs - 1) // bs for a, n in zip(starts, lens)]
    perm = rng.permutation(sum(per))
    slots, older, first = [], [], 0
    for a, n, p in zip(starts, lens, per):
        t = a + np.arange(n)
        slots.append(perm[first + t // bs] * bs + t % bs)
        older.append(perm[first] * bs + np.arange(a))
        first += p
    slots, older = np.concatenate(slots), np.concatenate(older)
    slots[rng.random(T) < 0.01] = -1
    pool = kvq.KVPool(first, bs, hkv, d, FMT, device=DEV)
    ref = Fp4Cache(first, bs, hkv, d)
    for at in (older, slots):
        k, v = _rows(rng, len(at), hkv, d), _rows(rng, len(at), hkv, d)
        if len(at) == 0:
            continue
        if way == "fused":
            pool.rope_append(None, None, _t(k), _t(v), None, _t(at))
        elif way == "strided":
            wide = _t(np.concatenate([k, v], 1))
            kvq.kvq_append_strided(pool.handle, wide[:, :hkv], wide[:, hkv:], _t(at))
        else:
            pool.append(_t(k), _t(v), _t(at))
        ref.append(k, v, at)
    assert pool.error() == kvq.KVQ_OK
    at = np.unique(np.concatenate([older, slots]))
    _check(pool, ref, at[at >= 0])
    pool.close()


def test_reads_of_many_slots():
    """Long read-backs: runs, single slots in any order, the same slot twice, padding (whose
    rows stay) and slots outside the pool (flagged)."""
    rng = np.random.default_rng(3)
    bs, hkv, d, nb = 32, 3, 64, 90
    pool = kvq.KVPool(nb, bs, hkv, d, FMT, device=DEV)
    ref = Fp4Cache(nb, bs, hkv, d)
    at = np.arange(nb * bs)
    k, v = _rows(rng, len(at), hkv, d), _rows(rng, len(at), hkv, d)
    pool.append(_t(k), _t(v), _t(at))
    ref.append(k, v, at)
    ask = np.concatenate([at[5:1500], rng.integers(0, nb * bs, 300), [-1] * 5, at[100:117], at[200:190:-1], [7] * 20, at[1501:], [-3]])
    for bad in (False, True):
        if bad:
            ask[[3, 700, 1600]] = nb * bs, 1 << 50, nb * bs + 9
        ko, vo = (torch.full((len(ask), hkv, d), 7.0, dtype=torch.float16, device=DEV) for _ in range(2))
        kvq.kvq_read_values(pool.handle, _t(ask), ko, vo)
        assert pool.error() == (kvq.KVQ_ERR_OUT_OF_RANGE if bad else kvq.KVQ_OK)
        real = (ask >= 0) & (ask < nb * bs)
        want = ref.values(ask[real])
        for got, x in ((ko, 0), (vo, 1)):
            got = got.cpu().numpy()
            np.testing.assert_array_equal(got[real], want[:, x].astype(np.float16))
            assert (got[~real] == 7).all()
    pool.close()


@pytest.mark.parametrize("T", [48, 1100])
def test_bad_slots_are_flagged_and_skipped(T):
    rng = np.random.default_rng(T)
    pool = kvq.KVPool(100, 16, 1, 64, FMT, device=DEV)
    ref = Fp4Cache(100, 16, 1, 64)
    slots = np.arange(T, dtype=np.int64)
    slots[5], slots[17], slots[33] = 1600, -7, 1 << 40
    k, v = _rows(rng, T, 1, 64), _rows(rng, T, 1, 64)
    pool.append(_t(k), _t(v), _t(slots))
    ref.append(k, v, slots)
    assert pool.error() == kvq.KVQ_ERR_OUT_OF_RANGE and pool.error() == kvq.KVQ_OK
    _check(pool, ref, np.setdiff1d(np.arange(T), [5, 17, 33]))
    pool.close()


@pytest.mark.parametrize("way", ["append", "fused"])
@pytest.mark.parametrize("T", [256, 2048])
def test_codes_at_the_borders(way, T):
    """Values on and next to the codes' and the scales' borders, every scale, zero groups,
    infinities and NaN: the bits of the definition, by the short and the long form."""
    rng = np.random.default_rng(12)
    hkv, d, bs = 1, 128, 16
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 0, 0.5, 1, 1.5, 2, 3, 4, 5.5])
    s = SCALES[rng.integers(0, len(SCALES), (T, hkv, 8, 1))]
    x = ties[rng.integers(0, 16, (T, hkv, 8, 16))] * s
    x[..., 0] = (6 * s)[..., 0]  # absmax: the scale is exactly s
    x[::5] *= 1 + rng.random((len(x[::5]), hkv, 8, 16)) / 3  # and next to everything
    x[1::5, ..., 0] = (6 * (s + SCALES[rng.integers(0, len(SCALES), s.shape)] / 16))[1::5, ..., 0]
    x = np.clip(x * rng.choice([-1, 1], x.shape), -65504, 65504).reshape(T, hkv, d).astype(np.float16)
    near = rng.random(x.shape) < 0.3  # fp16 neighbours of the borders
    x[near] = np.nextafter(x[near], np.float16(0))
    x[3] = 0
    x[4] = -0.0
    x[6, 0, 17], x[6, 0, 40], x[7, 0, 3], x[7, 0, 70:90] = np.nan, np.inf, -np.inf, np.nan
    x[8] = np.nan
    x[9] = 65504
    slots = np.arange(T, dtype=np.int64)
    pool = kvq.KVPool(T // bs, bs, hkv, d, FMT, device=DEV)
    ref = Fp4Cache(T // bs, bs, hkv, d)
    if way == "append":
        pool.append(_t(x), _t(-x), _t(slots))
    else:
        pool.rope_append(None, None, _t(x), _t(-x), None, _t(slots))
    ref.append(x, -x, slots)
    _check(pool, ref, slots)
    pool.close()


@pytest.mark.parametrize("T", [496, 3968])
def test_the_scale_of_every_absmax(T):
    """Every finite fp16 value as a group's largest (all 31744, or the 3968 smallest), by the
    long and the short form."""
    x = np.random.default_rng(4).uniform(-1, 1, (T * 8, 16))
    x[:, 5] = -1
    x = x * np.arange(T * 8, dtype=np.uint16).view(np.float16).astype(np.float64)[:, None]
    x = x.astype(np.float16).reshape(T, 1, 128)
    slots = np.arange(T, dtype=np.int64)
    pool = kvq.KVPool(T // 16, 16, 1, 128, FMT, device=DEV)
    ref = Fp4Cache(T // 16, 16, 1, 128)
    pool.append(_t(x), _t(x[:, :, ::-1]), _t(slots))
    ref.append(x, x[:, :, ::-1], slots)
    _check(pool, ref, slots)
    pool.close()


def test_values_beyond_fp16_saturate():
    """bf16 rows reach 3e38: the largest scale, the largest code."""
    x = torch.randn((32, 1, 64), device=DEV).bfloat16()
    x[3] *= 1e30
    pool = kvq.KVPool(2, 16, 1, 64, FMT, device=DEV)
    at = torch.arange(32, device=DEV)
    pool.rope_append(None, None, x, x, None, at)
    ref = Fp4Cache(2, 16, 1, 64)
    ref.append(x.float().cpu().numpy(), x.float().cpu().numpy(), at.cpu().numpy())
    _check(pool, ref, np.arange(32))
    assert pool.read_values(at)[0].abs().max() == 61440
    pool.close()


@pytest.mark.parametrize("T,bs,d", [(37, 16, 128), (2100, 32, 64)])
def test_rotated_append(T, bs, d):
    """Keys quantized from the fp32 rotation: the reference's code, or, where the float64
    quotient lies within the rotation's error (2^-19 of the pair's length) of a border,
    its neighbour."""
    rng = np.random.default_rng(T)
    hq, hkv = 4, 2
    plan = kvq.kvq_rope_init(d)
    pos = rng.integers(0, 100000, T)
    w = (1 + 0.1 * rng.standard_normal(d)).astype(np.float32)
    q, k, v = _rows(rng, T, hq, d), _rows(rng, T, hkv, d), _rows(rng, T, hkv, d)
    pool = kvq.KVPool(-(-T // bs), bs, hkv, d, FMT, device=DEV)
    at = np.arange(T)
    got = pool.rope_append(plan, _t(q), _t(k), _t(v), _t(pos), _t(at), k_weight=_t(w))
    codes, scales = (x.cpu().numpy() for x in pool.read_slots(_t(at)))
    y = rope(k, pos, frequencies(d), weight=w, eps=1e-6)
    vc, vs = quantize(v)
    np.testing.assert_array_equal(codes[:, 1], vc)
    np.testing.assert_array_equal(scales[:, 1], SCALES[vs].astype(np.float32))
    want, sb = quantize(y.astype(np.float32))
    off = (scales[:, 0] != SCALES[sb].astype(np.float32)).mean()
    assert off < 1e-3  # (a border within 2^-19 is met by chance)
    same = (scales[:, 0] == SCALES[sb].astype(np.float32)).repeat(16, -1)
    assert ((codes[:, 0] != want) & same).mean() < 1e-4
    val = np.asarray(values(codes[:, 0], nearest_bytes(scales[:, 0])))
    assert np.abs(val - y).max() <= np.abs(y).max() / 5
    np.testing.assert_allclose(got.float().cpu().numpy(), rope(q, pos, frequencies(d)), rtol=2.0 ** -10, atol=2.0 ** -8)
    pool.close()


def nearest_bytes(s):
    return np.searchsorted(SCALES, s.astype(np.float64)).astype(np.uint8)


# ------------------------------------------------------------------ single tokens
SHAPES = [(16, 8, 2, 128, [1, 0, 17, 333, 16, 900]), (32, 4, 1, 64, [31, 33, 500, 64]), (64, 6, 2, 64, [63, 65, 1, 700]),
          (64, 4, 4, 128, [129, 0, 640]), (16, 24, 2, 128, [45, 400]), (16, 32, 1, 64, [250]), (32, 3, 3, 128, [200, 64]),
          (16, 5, 1, 128, [48, 47, 49, 15, 80]), (16, 8, 8, 64, [100] * 9 + [3]), (16, 2, 1, 64, [1])]


@pytest.mark.parametrize("bs,hq,hkv,d,lens", SHAPES)
def test_decode(bs, hq, hkv, d, lens):
    pool, ref, table, lens, rng = _filled(bs, hkv, d, lens, seed=bs + hq)
    q = rng.standard_normal((len(lens), hq, d)).astype(np.float16)
    want, want_lse, weights = ref.attend(q, table, lens)
    most = int(max(lens.max(), 1))
    for split in (0, 1, 3, 5):
        out = pool.decode(_t(q), _t(table), _t(lens), most, split_blocks=split)
        assert pool.error() == kvq.KVQ_OK
        _near(out.cpu().numpy(), want)
    wide_q = torch.zeros((len(lens), hq + 3, d), dtype=torch.float16, device=DEV)
    wide_q[:, 2:2 + hq] = _t(q)
    wide = torch.full((len(lens), hq + 1, d), 9.0, device=DEV)
    ws = torch.empty(kvq.kvq_decode_workspace_bytes(pool.handle, len(lens), hq, most), dtype=torch.uint8, device=DEV)
    kvq.kvq_paged_decode_strided(pool.handle, wide_q[:, 2:2 + hq], _t(table), _t(lens), most, d ** -0.5, wide[:, 1:], ws)
    _near(wide[:, 1:].cpu().numpy(), want)
    assert (wide[:, 0] == 9).all()
    out = torch.empty((len(lens), hq, d), device=DEV)
    kvq.kvq_paged_decode_noalloc(pool.handle, _t(q), _t(table), _t(lens), most, d ** -0.5, out)
    _near(out.cpu().numpy(), want)
    # log-sum-exps, and the weights they give (2^-14: |z| <= 16 within 2^-21, twice)
    out, lse = pool.decode_lse(_t(q), _t(table), _t(lens), most)
    _near(out.cpu().numpy(), want)
    np.testing.assert_allclose(lse.cpu().numpy(), want_lse, rtol=2.0 ** -18, atol=2.0 ** -16)
    scores = torch.zeros((len(lens), hkv, most), device=DEV)
    pool.accumulate_weights(_t(q), _t(table), _t(lens), most, lse, scores)
    for s in range(len(lens)):
        got = scores[s].cpu().numpy()
        assert (got[:, lens[s]:] == 0).all()
        if lens[s]:
            np.testing.assert_allclose(got[:, :lens[s]], weights[s].sum(1), rtol=2.0 ** -14, atol=1e-9)
    assert pool.error() == kvq.KVQ_OK
    pool.close()


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_softmax_scales(scale):
    """Uniform weights, reversed ones, and ones that all but a few tokens lose."""
    pool, ref, table, lens, rng = _filled(16, 2, 128, [70, 200, 5], seed=3)
    q = rng.standard_normal((3, 8, 128)).astype(np.float16)
    out = pool.decode(_t(q), _t(table), _t(lens), 200, sm_scale=scale)
    # scores up to 2^7 in magnitude: weights within 2^-21 * 2^7 * 1.5 of themselves
    np.testing.assert_allclose(out.cpu().numpy(), ref.decode(q, table, lens, scale), rtol=0, atol=2e-3)
    assert torch.isfinite(out).all()
    pool.close()


@pytest.mark.parametrize("bs", [16, 32, 64])
def test_absent_blocks_are_skipped(bs):
    """Block ids outside the pool, at the start, inside and at the end of a row."""
    pool, ref, table, lens, rng = _filled(bs, 2, 128, [8 * bs + 3, 70, 5 * bs], seed=6)
    q = rng.standard_normal((3, 8, 128)).astype(np.float16)
    bad = table.copy()
    bad[0, [0, 3, 8]] = -1, 1 << 30, ref.blocks
    bad[2, :] = -5
    out = pool.decode(_t(q), _t(bad), _t(lens), int(lens.max()))
    assert pool.error() == kvq.KVQ_ERR_OUT_OF_RANGE
    assert torch.isfinite(out).all()
    keep = [t for t in range(lens[0]) if t // bs not in (0, 3, 8)]
    one = ref.values(tokens(table, lens, 0, bs)[keep])
    from cache_ops_ref import attention
    _near(out[0].cpu().numpy(), attention(lambda s: one, q[:1], [len(keep)])[0][0])
    _near(out[1].cpu().numpy(), ref.decode(q[1:2], table[1:2], lens[1:2])[0])
    assert (out[2] == 0).all()
    pool.close()


@pytest.mark.parametrize("bs", [16, 64])
def test_decode_steps(bs):
    """Steps that fill a block and start the next, the token appended by the call itself."""
    hq, hkv, d = 8, 2, 128
    pool, ref, table, lens, rng = _filled(bs, hkv, d, [bs - 2, 5 * bs - 1, 3], seed=1, spare=8)
    spare = np.setdiff1d(np.arange(ref.blocks), table.ravel())
    for s in range(3):
        table[s, (lens[s] + bs - 1) // bs] = spare[s]
    for _ in range(4):
        lens += 1
        k, v = _rows(rng, 3, hkv, d), _rows(rng, 3, hkv, d)
        q = rng.standard_normal((3, hq, d)).astype(np.float16)
        out = pool.decode_step(_t(k), _t(v), _t(q), _t(table), _t(lens), int(lens.max()))
        ref.append(k, v, [tokens(table, lens, s, bs)[-1] for s in range(3)])
        assert pool.error() == kvq.KVQ_OK
        _near(out.cpu().numpy(), ref.decode(q, table, lens))
    _check(pool, ref, np.concatenate([tokens(table, lens, s, bs) for s in range(3)]))
    k, v = _rows(rng, 3, hkv, d), _rows(rng, 3, hkv, d)
    bad = table.copy()
    bad[1, 0] = -1
    before = pool.buffer[256:].clone()
    pool.decode_step(_t(k), _t(v), _t(q), _t(bad), _t(np.array([0, 1, 0], np.int32)), bs)
    assert pool.error() == kvq.KVQ_ERR_OUT_OF_RANGE
    assert torch.equal(before, pool.buffer[256:])
    pool.close()


@pytest.mark.parametrize("bs", [16, 32, 64])
def test_cascade_prefill_and_copies(bs):
    hq, hkv, d = 8, 2, 128
    pool, ref, table, lens, rng = _filled(bs, hkv, d, [3 * bs + 5, 4 * bs, 2 * bs, bs - 1], seed=2, spare=9)
    table[1:3, :2] = table[0, :2]
    table[3, 0] = table[0, 0]
    S = 4
    q = rng.standard_normal((S, hq, d)).astype(np.float16)
    for prefix in (1, 2, 3):
        if prefix == 3:
            table[1:3, 2] = table[0, 2]
        out = pool.cascade_decode(_t(q), _t(table), _t(lens), int(lens.max()), prefix)
        np.testing.assert_allclose(out.cpu().numpy(), ref.decode(q, table, lens), rtol=0, atol=TOL)
    spare = np.setdiff1d(np.arange(ref.blocks), table.ravel())[:2].astype(np.int32)
    kvq.kvq_copy_blocks(pool.handle, _t(table[1, :2]), _t(spare))
    own = table.copy()
    own[1, :2] = spare
    a = pool.decode(_t(q), _t(table), _t(lens), int(lens.max()))
    b = pool.decode(_t(q), _t(own), _t(lens), int(lens.max()))
    assert torch.equal(a, b)
    n = [bs + 3, 1, 2 * bs, bs - 1]
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    qq = rng.standard_normal((start[-1], hq, d)).astype(np.float16)
    want = np.concatenate([ref.decode(qq[start[s]:start[s + 1]], np.repeat(table[s:s + 1], n[s], 0),
                                      np.arange(lens[s] - n[s], lens[s]) + 1) for s in range(S)])
    for two in (False, True):
        got = torch.zeros((int(start[-1]), hq, d), device=DEV)
        if two:
            ws = torch.full((kvq.kvq_prefill_workspace_bytes(pool.handle, S, int(lens.max())),), 0xFF, dtype=torch.uint8, device=DEV)
            assert ws.numel()
            kvq.kvq_prefill_ex(pool.handle, _t(qq), _t(start), max(n), _t(table), _t(lens), int(lens.max()), d ** -0.5, got, ws)
        else:
            kvq.kvq_prefill(pool.handle, _t(qq), _t(start), max(n), _t(table), _t(lens), int(lens.max()), d ** -0.5, got)
        _near(got.cpu().numpy(), want)
    assert pool.error() == kvq.KVQ_OK
    pool.close()


@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (64, 12, 1), (128, 4, 4)])
def test_prefill_shapes(d, hq, hkv):
    bs, lens = 16, [70, 129, 1]
    pool, ref, table, lens, rng = _filled(bs, hkv, d, lens, seed=d + hq)
    start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    qq = rng.standard_normal((start[-1], hq, d)).astype(np.float16)
    want = np.concatenate([ref.decode(qq[start[s]:start[s + 1]], np.repeat(table[s:s + 1], lens[s], 0), np.arange(lens[s]) + 1)
                           for s in range(len(lens))])
    ws = torch.empty(kvq.kvq_prefill_workspace_bytes(pool.handle, 3, 129), dtype=torch.uint8, device=DEV)
    got = torch.empty((int(start[-1]), hq, d), device=DEV)
    kvq.kvq_prefill_ex(pool.handle, _t(qq), _t(start), 129, _t(table), _t(lens), 129, d ** -0.5, got, ws)
    _near(got.cpu().numpy(), want)
    kvq.kvq_prefill(pool.handle, _t(qq), _t(start), 129, _t(table), _t(lens), 129, d ** -0.5, got)
    _near(got.cpu().numpy(), want)
    pool.close()


def test_step_captured_in_a_graph():
    """A captured append + step replays on what the buffers hold then."""
    bs, hq, hkv, d = 16, 4, 1, 64
    pool, ref, table, lens, rng = _filled(bs, hkv, d, [20, 40], seed=4)
    kb, vb = torch.empty((2, hkv, d), dtype=torch.float16, device=DEV), torch.empty((2, hkv, d), dtype=torch.float16, device=DEV)
    q, L = _t(rng.standard_normal((2, hq, d)).astype(np.float16)), _t(lens)
    tb, out = _t(table), torch.empty((2, hq, d), device=DEV)
    ws = torch.empty(kvq.kvq_decode_workspace_bytes(pool.handle, 2, hq, 48), dtype=torch.uint8, device=DEV)
    kvq.kvq_paged_decode(pool.handle, q, tb, L, 48, d ** -0.5, out, ws)
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


def test_blocks_beyond_four_gigabytes():
    bs, hkv, d = 16, 8, 128
    nb = (5 << 30) // (2304 * hkv)
    pool = kvq.KVPool(nb, bs, hkv, d, FMT, device=DEV)
    rng = np.random.default_rng(8)
    blocks = np.array([nb - 1, 3, nb - 7, nb // 2])
    at = (blocks[:, None] * bs + np.arange(bs)).reshape(-1)
    k, v = _rows(rng, 64, hkv, d), _rows(rng, 64, hkv, d)
    pool.append(_t(k), _t(v), _t(at))
    kq, ks = quantize(k)
    vq, vs = quantize(v)
    codes, scales = pool.read_slots(_t(at))
    np.testing.assert_array_equal(codes.cpu().numpy(), np.stack([kq, vq], 1))
    kv, vv = values(kq, ks), values(vq, vs)
    q = rng.standard_normal((1, 8, d)).astype(np.float16)
    out = pool.decode(_t(q), _t(blocks[None].astype(np.int32)), _t(np.array([61], np.int32)), 64)
    from cache_ops_ref import attention
    _near(out.cpu().numpy(), attention(lambda s: np.stack([kv, vv], 1)[:61], q, [61])[0])
    pool.close()


@pytest.mark.parametrize("hq", [4, 8])
def test_long_range_in_one_warp_does_not_drift(hq):
    """24000 tokens summed by one warp: the sum stays in fp32 adds."""
    pool, ref, table, lens, rng = _filled(16, 1, 128, [24000], seed=5)
    q = rng.standard_normal((1, hq, 128)).astype(np.float16)
    out = pool.decode(_t(q), _t(table), _t(lens), 24000, split_blocks=1500)
    _near(out.cpu().numpy(), ref.decode(q, table, lens))
    pool.close()


def test_a_wait_that_runs_out():
    """A page copy that never comes: flagged, the next decode is right."""
    pool, ref, table, lens, rng = _filled(16, 2, 128, [300, 70], seed=7)
    q = rng.standard_normal((2, 8, 128)).astype(np.float16)
    ws = torch.empty(kvq.kvq_decode_workspace_bytes(pool.handle, 2, 8, 300), dtype=torch.uint8, device=DEV)
    out = torch.empty((2, 8, 128), device=DEV)
    kvq.kvq_selftest_decode_timeout(pool.handle, _t(q), _t(table), _t(lens), 300, out, ws, wait_tries=5)
    assert pool.error() == kvq.KVQ_ERR_TIMEOUT
    kvq.kvq_paged_decode(pool.handle, _t(q), _t(table), _t(lens), 300, 128 ** -0.5, out, ws)
    assert pool.error() == kvq.KVQ_OK
    _near(out.cpu().numpy(), ref.decode(q, table, lens))
    pool.close()


@pytest.mark.parametrize("fmt", [FMT, kvq.KVQ_INT8_PER_BLOCK])
@pytest.mark.parametrize("S,hq", [(2048, 1), (2049, 1), (2048, 4), (2049, 4)])
def test_many_sequences(fmt, S, hq):
    """As many sequences as the merge counts itself, and one more (one head), and so many
    rows that the merge of many takes them (four heads); a few long ones that are cut, so
    that pieces are joined.  Rows drawn from all over against float64."""
    rng = np.random.default_rng(S)
    bs, hkv, d = 16, 1, 64
    lens = rng.integers(0, 12, S).astype(np.int32)
    lens[[0, 700, S - 1]] = 3000, 1777, 2500
    per = -(-lens // bs)
    table = np.zeros((S, int(per.max())), np.int32)
    at = np.concatenate([[0], np.cumsum(per)])
    for s in range(S):
        table[s, :per[s]] = np.arange(at[s], at[s + 1])
    slots = np.concatenate([tokens(table, lens, s, bs) for s in range(S)])
    pool = kvq.KVPool(int(at[-1]), bs, hkv, d, fmt, device=DEV)
    pool.append(_t(_rows(rng, len(slots), hkv, d)), _t(_rows(rng, len(slots), hkv, d)), _t(slots))
    q = rng.standard_normal((S, hq, d)).astype(np.float16)
    out = pool.decode(_t(q), _t(table), _t(lens), 3000).cpu().numpy()
    pick = np.unique(np.concatenate([[0, 1, 699, 700, 701, S - 2, S - 1], rng.integers(0, S, 30)]))
    codes, scales = (x.double().cpu().numpy() for x in pool.read_slots(_t(slots)))
    held = np.zeros((int(at[-1]) * bs, 2, hkv, d))
    if fmt == FMT:
        held[slots] = values(codes.astype(np.uint8), nearest_bytes(scales))
    else:
        held[slots] = codes * scales[..., None]
    want = attention(lambda i: held[tokens(table, lens, pick[i], bs)], q[pick], lens[pick])[0]
    _near(out[pick], want)
    pool.close()
