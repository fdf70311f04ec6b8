"""kvq_rope against float64: layouts, partly rotated heads, scalings, far and
negative positions, norms, types, strides, in place; kvq_rope_append against the
same rotation followed by each format's own quantizer."""
import numpy as np
import pytest
import torch

import oracle
import paged_quantized_kv_kvq_gb300 as kvq
from cache_ops_ref import BlockCache, frequencies, rope, rope_bound

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
SCALINGS = {kvq.KVQ_ROPE_NONE: {}, kvq.KVQ_ROPE_LINEAR: dict(factor=4.0), kvq.KVQ_ROPE_BASE: dict(factor=8.0),
            kvq.KVQ_ROPE_PARTS: dict(factor=16.0, orig_len=4096.0, low=1.0, high=32.0),
            kvq.KVQ_ROPE_BANDS: dict(factor=8.0, orig_len=8192.0, low=1.0, high=4.0)}


def _t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _rows(rng, T, h, d, dtype=torch.float16):
    x = rng.standard_normal((T, h, d)).astype(np.float32)
    x[..., ::31] *= 12
    return torch.from_numpy(x).to(dtype).to(DEV)


def _reference(x, positions, r, interleaved, scaling, weight, eps):
    f = frequencies(r, scaling=scaling, **SCALINGS[scaling]) if r else None
    m = 0.1 * np.log(16.0) + 1.0 if scaling == kvq.KVQ_ROPE_PARTS else 1.0
    x = x.float().cpu().numpy()
    w = None if weight is None else weight.cpu().numpy()
    y = rope(x, positions, f, interleaved, m, w, eps)
    return y, rope_bound(y, rope(x, weight=w, eps=eps), r, interleaved, m)


def _within(got, want, bound):
    d = np.abs(got.cpu().numpy().astype(np.float64) - want)
    assert (d <= bound).all(), (d - bound).max()


@pytest.mark.parametrize("T,hq,hk,d,r", [(1, 4, 1, 64, 64), (7, 32, 8, 128, 128), (3, 5, 3, 128, 64),
                                         (33, 12, 2, 64, 16), (600, 6, 2, 128, 96), (4099, 3, 1, 64, 32),
                                         (2, 1, 0, 128, 32), (5, 0, 7, 64, 48), (1, 71, 1, 128, 112)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,dtype", [(True, torch.float16), (False, torch.bfloat16), (True, torch.bfloat16)])
def test_rope(T, hq, hk, d, r, interleaved, norm, dtype):
    rng = np.random.default_rng(T * 7 + hq)
    q = _rows(rng, T, hq, d, dtype) if hq else None
    k = _rows(rng, T, hk, d, dtype) if hk else None
    pos = rng.integers(-5000, 1 << 20, T)
    qw = _t(rng.standard_normal(d).astype(np.float32)) if norm else None
    kw = _t(rng.standard_normal(d).astype(np.float32)) if norm and T % 2 else None
    plan = kvq.kvq_rope_init(r, interleaved)
    qo = torch.empty((T, hq, d), dtype=torch.float16, device=DEV) if hq else None
    ko = torch.empty((T, hk, d), dtype=torch.float16, device=DEV) if hk else None
    kvq.kvq_rope(plan, q, k, _t(pos), qo, ko, qw, kw, 1e-5)
    for x, o, w in ((q, qo, qw), (k, ko, kw)):
        if x is not None:
            _within(o, *_reference(x, pos, r, interleaved, kvq.KVQ_ROPE_NONE, w, 1e-5))


@pytest.mark.parametrize("scaling", list(SCALINGS))
def test_scalings_and_far_positions(scaling):
    rng = np.random.default_rng(scaling)
    pos = np.array([0, 1, 4095, 131071, (1 << 31) + 12345, (1 << 40) - 1, -7], np.int64)
    q = _rows(rng, len(pos), 2, 128)
    plan = kvq.kvq_rope_init(128, scaling=scaling, **SCALINGS[scaling])
    out = torch.empty_like(q)
    kvq.kvq_rope(plan, q, None, _t(pos), out)
    _within(out, *_reference(q, pos, 128, False, scaling, None, 0.0))


@pytest.mark.parametrize("T", [5, 700, 5000])
def test_strides_and_in_place(T):
    """Views of packed rows, outputs into wider rows, and rows turned where they lie:
    the same bits each time, and nothing outside the rows written."""
    rng = np.random.default_rng(T)
    hq, hk, d = 6, 2, 128
    qkv = _rows(rng, T, hq + 2 * hk, d)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    pos = _t(rng.integers(0, 100000, T))
    plan = kvq.kvq_rope_init(64, True)
    qo, ko = torch.empty((T, hq, d), dtype=torch.float16, device=DEV), torch.empty((T, hk, d), dtype=torch.float16, device=DEV)
    kvq.kvq_rope(plan, q.contiguous(), k.contiguous(), pos, qo, ko)
    wide = torch.full((T, hq + hk + 3, d), 9.0, dtype=torch.float16, device=DEV)
    kvq.kvq_rope(plan, q, k, pos, wide[:, 1:1 + hq], wide[:, 2 + hq:2 + hq + hk])
    assert torch.equal(wide[:, 1:1 + hq], qo) and torch.equal(wide[:, 2 + hq:2 + hq + hk], ko)
    assert (wide[:, 0] == 9).all() and (wide[:, 1 + hq] == 9).all() and (wide[:, -1] == 9).all()
    v = qkv[:, hq + hk:].clone()
    kvq.kvq_rope(plan, q, k, pos)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, hq + hk:], v)


def test_norm_alone_and_empty_calls():
    rng = np.random.default_rng(1)
    q = _rows(rng, 9, 3, 64, torch.bfloat16)
    w = _t(rng.standard_normal(64).astype(np.float32))
    out = torch.empty((9, 3, 64), dtype=torch.float16, device=DEV)
    kvq.kvq_rope(None, q, None, None, out, q_weight=w, eps=1e-6)
    _within(out, *_reference(q, None, 0, False, 0, w, 1e-6))
    out.fill_(3)
    kvq.kvq_rope(None, q[:0], None, None, out[:0])
    assert (out == 3).all()
    # a row of zeros stays zeros (eps > 0)
    z = torch.zeros((2, 3, 64), dtype=torch.float16, device=DEV)
    kvq.kvq_rope(None, z, None, None, out[:2], q_weight=w, eps=1e-6)
    assert (out[:2] == 0).all()


def test_side_stream_and_graph():
    rng = np.random.default_rng(2)
    q = _rows(rng, 8, 4, 128)
    pos = torch.zeros(8, dtype=torch.int64, device=DEV)
    plan = kvq.kvq_rope_init(128)
    out = torch.empty_like(q)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        kvq.kvq_rope(plan, q, None, pos, out)
    plan2 = kvq.kvq_rope_init(128, True)  # the captured call keeps its own plan
    del plan
    for p in (5, 100000):
        pos.fill_(p)
        g.replay()
        torch.cuda.synchronize()
        _within(out, *_reference(q, [p] * 8, 128, False, 0, None, 0.0))
    assert plan2.rotary_dim == 128
    # an explicit stream orders the call
    with torch.cuda.stream(side):
        big = torch.randn(1 << 24, device=DEV).sum()
        pos2 = torch.full((8,), 77, device=DEV)
    kvq.kvq_rope(plan2, q, None, pos2, out, stream=side)
    side.synchronize()
    _within(out, *_reference(q, [77] * 8, 128, True, 0, None, 0.0))
    assert torch.isfinite(big)


# ------------------------------------------------------------------ fused with the append
FORMATS = [(kvq.KVQ_FP16, 0), (kvq.KVQ_INT8_PER_TOKEN, 0), (kvq.KVQ_INT8_PER_CHANNEL, 0), (kvq.KVQ_INT8_PER_GROUP, 128),
           (kvq.KVQ_INT8_PER_GROUP, 16), (kvq.KVQ_FP8_E4M3_PER_TOKEN, 0), (kvq.KVQ_INT4_PER_GROUP, 32),
           (kvq.KVQ_FP8_E5M2, 0), (kvq.KVQ_INT8_PER_BLOCK, 0), (kvq.KVQ_FP8_E4M3_PER_BLOCK, 0)]


def _slots(rng, lens, bs, starts):
    """Sequences of `lens` new tokens from positions `starts`, their blocks scattered."""
    per = [(a + n + bs - 1) // bs for a, n in zip(starts, lens)]
    perm = rng.permutation(sum(per))
    out, first = [], 0
    for n, p, a in zip(lens, per, starts):
        t = np.arange(a, a + n)
        out.append(perm[first + t // bs] * bs + t % bs)
        first += p
    return np.concatenate(out).astype(np.int64), sum(per)


def _plain_pool(fmt, group, nb, bs, hkv, d, chan):
    pool = kvq.KVPool(nb, bs, hkv, d, fmt, group, device=DEV)
    if fmt == kvq.KVQ_INT8_PER_CHANNEL:
        kvq.kvq_set_channel_scales(pool.handle, chan, chan)
    return pool


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("bs,hq,hkv,d,lens,starts,dtype", [
    (16, 8, 2, 128, [1, 1, 1, 1, 1], [0, 5, 15, 16, 40], torch.float16),     # decode steps
    (32, 3, 1, 64, [50, 1, 64, 33], [0, 9, 0, 0], torch.float16),
    (64, 4, 4, 128, [70, 200], [0, 0], torch.bfloat16),
    (16, 8, 2, 64, [700, 500, 17, 1], [0, 0, 3, 2], torch.bfloat16),         # many tokens, runs cut anywhere
    (8, 2, 3, 128, [11, 1], [0, 4], torch.float16), (8, 2, 1, 64, [1200], [0], torch.float16),
    (16, 20, 20, 128, [1, 1, 2, 1], [3, 0, 14, 20], torch.bfloat16),         # more heads than a CTA's rows
    (32, 40, 40, 64, [1] * 150, [s % 37 for s in range(150)], torch.float16),
    (16, 4, 2, 128, [1] * 1100 + [40, 16], [5] * 1100 + [0, 16], torch.float16)])  # a long call of single tokens
def test_rope_append(fmt, group, bs, hq, hkv, d, lens, starts, dtype):
    if bs == 8 and fmt == kvq.KVQ_INT4_PER_GROUP:
        pytest.skip("INT4 takes blocks of 16 tokens or more")
    if group > d:
        group = d
    rng = np.random.default_rng(bs * 100 + hq)
    T = sum(lens)
    slots, nb = _slots(rng, lens, bs, starts)
    qkv = _rows(rng, T, hq + 2 * hkv, d, dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    pos = rng.integers(0, 1 << 17, T)
    r, inter = d // 2, bool(bs & 16)
    plan = kvq.kvq_rope_init(r, inter)
    w = _t(1 + 0.1 * rng.standard_normal(d).astype(np.float32))
    chan = torch.full((hkv, d), 0.05, device=DEV)
    pool = _plain_pool(fmt, group, nb, bs, hkv, d, chan)
    qo = pool.rope_append(plan, q, k, v, _t(pos), _t(slots), q_weight=w, k_weight=w, eps=1e-6)
    assert pool.error() == kvq.KVQ_OK
    _within(qo, *_reference(q, pos, r, inter, 0, w, 1e-6))
    codes, scales = (None if x is None else x.cpu().numpy() for x in pool.read_slots(_t(slots)))
    # V has no arithmetic before its quantizer: bit for bit
    vv = v.float()
    y, _ = _reference(k, pos, r, inter, 0, w, 1e-6)
    if fmt in kvq.BLOCK_FORMATS:
        ref = BlockCache(fmt, nb, bs, hkv, d)
        ref.append(y.astype(np.float32), vv.cpu().numpy(), slots)
        rc, rs = ref.codes[slots], ref.scales[slots // bs]
    elif fmt == kvq.KVQ_FP16:
        rc, rs = np.stack([y, vv.cpu().numpy()], 1).astype(np.float16), None
    else:
        ref = oracle.OracleCache(fmt, nb, bs, hkv, d, group)
        ref.chan_scales[:] = 0.05
        ref.append(y.astype(np.float32), vv.cpu().numpy(), slots)
        rc, rs = ref.codes[slots], None if scales is None else ref.scales[slots]
    np.testing.assert_array_equal(np.ascontiguousarray(codes[:, 1]).view(np.uint8),
                                  np.ascontiguousarray(rc[:, 1].astype(codes.dtype)).view(np.uint8))
    if rs is not None:
        np.testing.assert_array_equal(scales[:, 1], rs[:, 1])
        # K scales.  A rotated value is off by at most (2^-20 + 2^-21) m (|u| + |v|), u and
        # v its pair before the rotation (rope_bound), which 2^-19 max|x| over the normed
        # head bounds (|u| + |v| <= 2 max|x|, less than 2^-19 max|x| * 2 * 3/4 in all); an
        # absmax moves by no more than its largest element, wherever v lies -- in another
        # group than u, for instance, so this is no bound relative to the scale itself.
        # The scale is that over the largest code, with one fp32 division (2^-24).
        top = 448 if fmt in (kvq.KVQ_FP8_E4M3_PER_TOKEN, kvq.KVQ_FP8_E4M3_PER_BLOCK) else 7 if fmt == kvq.KVQ_INT4_PER_GROUP else 127
        reach = np.abs(rope(k.float().cpu().numpy(), weight=w.cpu().numpy(), eps=1e-6)).max((1, 2))
        reach = np.full_like(reach, reach.max()) if fmt in kvq.BLOCK_FORMATS else reach
        bound = 1.5 * 2.0 ** -19 * reach / top
        assert (np.abs(scales[:, 0] - rs[:, 0].astype(np.float64)) <=
                bound.reshape(-1, *[1] * (rs.ndim - 2)) + 2.0 ** -23 * rs[:, 0]).all()
    # K codes: the same, or the neighbour where the value sits at a border.  Rounded
    # values a code apart at most, and only near borders: 2^-18 of the pair's length
    # relative to a step of 2^-7 absmax (2^-3 for INT4) leaves well under 1%.
    if fmt == kvq.KVQ_FP16:
        a, b = codes[:, 0].astype(np.float64), rc[:, 0].astype(np.float64)
        assert (np.abs(a - b) <= np.abs(b) * 2.0 ** -10 + 2.0 ** -18 * np.abs(y).max()).all()
    else:
        a, b = codes[:, 0], rc[:, 0].astype(codes.dtype)
        if a.dtype == np.uint8:  # sign-magnitude codes: neighbours differ by one
            a, b = (np.where(x & 0x80, -(x & 0x7F).astype(int), x.astype(int)) for x in (a, b))
        d_ = np.abs(a.astype(int) - b.astype(int))
        assert d_.max() <= 1 and (d_ > 0).mean() < 0.01
    pool.close()


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_without_rotation_it_is_the_append(fmt, group):
    """No plan, no norm, fp16 rows: the bits of kvq_append, token by token and whole."""
    rng = np.random.default_rng(6)
    bs, hkv, d = 16, 2, 128
    for lens in ([3, 17, 1], [900, 300]):
        slots, nb = _slots(rng, lens, bs, [0] * len(lens))
        k, v = _rows(rng, sum(lens), hkv, d), _rows(rng, sum(lens), hkv, d)
        chan = torch.full((hkv, d), 0.05, device=DEV)
        a, b = _plain_pool(fmt, group, nb, bs, hkv, d, chan), _plain_pool(fmt, group, nb, bs, hkv, d, chan)
        pad = slots.copy()
        pad[::50] = -1 if fmt not in kvq.BLOCK_FORMATS else pad[::50]
        a.append(k, v, _t(pad))
        assert b.rope_append(None, None, k, v, None, _t(pad)) is None
        keep = pad[pad >= 0]
        for x, y in zip(a.read_slots(_t(keep)), b.read_slots(_t(keep))):
            assert x is None or torch.equal(x, y)
        a.close()
        b.close()


@pytest.mark.parametrize("fmt,group", [(kvq.KVQ_INT8_PER_BLOCK, 0), (kvq.KVQ_INT8_PER_GROUP, 128)])
@pytest.mark.parametrize("graph", [False, True])
def test_long_append_and_the_step_behind_it(fmt, group, graph):
    """A prompt long enough for two kernels, and right behind it on the stream a step
    whose append launches as a programmatic dependent: eagerly and replayed, the
    same as with a synchronisation between the two."""
    rng = np.random.default_rng(21)
    bs, hq, hkv, d, S = 16, 8, 2, 128, 3
    lens = [900, 700, 555]
    slots, nb = _slots(rng, lens, bs, [0] * S)
    T = sum(lens)
    qkv = _rows(rng, T, hq + 2 * hkv, d)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    pos = _t(np.concatenate([np.arange(n) for n in lens]))
    per = [(n + bs - 1) // bs for n in lens]
    table = np.zeros((S, max(per) + 1), np.int32)
    at = 0
    spare = nb
    for s, n in enumerate(lens):
        table[s, :per[s]] = slots[at:at + n:bs] // bs
        table[s, per[s]] = spare  # (the step may need a new block)
        spare += 1
        at += n
    L = _t(np.array(lens, np.int32) + 1)
    plan = kvq.kvq_rope_init(d)
    kn, vn, qn = (_rows(rng, S, h, d) for h in (hkv, hkv, hq))
    results = []
    for apart in (True, False):
        pool = kvq.KVPool(spare, bs, hkv, d, fmt, group, device=DEV)
        qo, out = torch.empty((T, hq, d), dtype=torch.float16, device=DEV), torch.zeros((S, hq, d), device=DEV)
        ws = torch.empty(kvq.kvq_decode_workspace_bytes(pool.handle, S, hq, 901), dtype=torch.uint8, device=DEV)
        sl, tb = _t(slots), _t(table)

        def call():
            kvq.kvq_rope_append(pool.handle, plan, q, k, v, pos, sl, qo)
            if apart:
                torch.cuda.synchronize()
            kvq.kvq_decode_step(pool.handle, kn, vn, qn, tb, L, 901, d ** -0.5, out, ws)

        call()
        torch.cuda.synchronize()
        if graph and not apart:
            g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
            with torch.cuda.graph(g, stream=side):
                call()
            for _ in range(5):
                out.zero_()
                g.replay()
                torch.cuda.synchronize()
        for _ in range(0 if graph else 5):
            call()
        torch.cuda.synchronize()
        assert pool.error() == kvq.KVQ_OK
        results.append((qo.clone(), out.clone()) + tuple(pool.read_slots(sl)))
        pool.close()
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_padding_and_bad_slots():
    """A padded token's queries are computed; a slot outside the pool is flagged."""
    rng = np.random.default_rng(8)
    for fmt in (kvq.KVQ_INT8_PER_GROUP, kvq.KVQ_INT8_PER_BLOCK, kvq.KVQ_FP8_E4M3_PER_TOKEN):
        pool = kvq.KVPool(2, 16, 1, 64, fmt, 64, device=DEV)
        before = pool.buffer[256:].clone()
        x = _rows(rng, 3, 3, 64)
        plan = kvq.kvq_rope_init(64)
        pos = np.array([4, 5, 6])
        qo = pool.rope_append(plan, x[:, :1], x[:, 1:2], x[:, 2:], _t(pos), _t(np.array([-1, -9, -1])))
        assert pool.error() == kvq.KVQ_OK and torch.equal(before, pool.buffer[256:])
        _within(qo, *_reference(x[:, :1], pos, 64, False, 0, None, 0.0))
        pool.rope_append(plan, x[:, :1], x[:, 1:2], x[:, 2:], _t(pos), _t(np.array([32, -1, 1 << 50])))
        assert pool.error() == kvq.KVQ_ERR_OUT_OF_RANGE and torch.equal(before, pool.buffer[256:])
        pool.close()


@pytest.mark.parametrize("which", ["q", "k", "positions", "q_out", "k_out", "q_weight", "k_weight"])
def test_tensors_of_another_device_are_refused(which):
    """Every tensor of a call is looked at, not the first alone."""

    class Elsewhere:
        """A tensor as another GPU would hold it."""

        def __init__(self, t):
            self.t = t

        is_cuda = True

        def __getattr__(self, name):
            return getattr(self.t, name)

        def get_device(self):
            return torch.cuda.current_device() + 1

    x = torch.zeros((2, 3, 64), dtype=torch.float16, device=DEV)
    a = dict(q=x, k=x.clone(), positions=torch.zeros(2, dtype=torch.int64, device=DEV), q_out=x.clone(), k_out=x.clone(),
             q_weight=torch.ones(64, device=DEV), k_weight=torch.ones(64, device=DEV))
    kvq.kvq_rope(kvq.kvq_rope_init(64), **a)
    a[which] = Elsewhere(a[which])
    with pytest.raises(ValueError):
        kvq.kvq_rope(kvq.kvq_rope_init(64), **a)


@pytest.mark.parametrize("fmt,group", [(kvq.KVQ_INT8_PER_BLOCK, 0), (kvq.KVQ_FP8_E4M3_PER_BLOCK, 0),
                                       (kvq.KVQ_INT8_PER_GROUP, 64), (kvq.KVQ_INT4_PER_GROUP, 32)])
@pytest.mark.parametrize("T", [200, 3000])
def test_a_slot_given_twice_spoils_its_own_block_only(fmt, group, T):
    rng = np.random.default_rng(T)
    nb, bs = T // 16 + 8, 16
    pools = [kvq.KVPool(nb, bs, 3, 64, fmt, group, device=DEV, fill_byte=0) for _ in range(2)]
    x = _rows(rng, T, 6, 64)
    slots = np.arange(T) + bs
    twice = slots.copy()
    twice[64:64 + 40] = slots[64]        # more tokens of one block than it holds
    twice[130:134] = slots[129]          # a few in the middle of a run
    for pool, at in zip(pools, (slots, twice)):
        pool.rope_append(None, None, x[:, :3], x[:, 3:], None, _t(at))
        assert pool.error() == kvq.KVQ_OK
    spoilt = np.unique(np.concatenate([slots[64:104], slots[129:134]]) // bs)
    rest = slots[~np.isin(slots // bs, spoilt)]
    rest = np.concatenate([np.arange(bs), rest, np.arange((T // bs + 3) * bs, nb * bs)])
    for a, b in zip(*(pool.read_values(_t(rest)) for pool in pools)):
        assert torch.equal(a, b)
    for pool in pools:
        pool.close()
