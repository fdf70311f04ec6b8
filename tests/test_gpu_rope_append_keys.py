"""Keys that kvq_rope_append stores, against the rotation in float64 followed by each
format's quantizer: rotary dimension and pair layout independent of the block size,
whole blocks, ragged runs and single tokens, every pool format."""
import numpy as np
import pytest
import torch

import oracle
import paged_quantized_kv_kvq_gb300 as kvq
from cache_ops_ref import BlockCache, frequencies, rope
from test_gpu_rope import FORMATS, _plain_pool, _rows, _slots, _t

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
EPS = 1e-6


def _values(fmt, group, codes, scales, chan):
    """float64 values of read_slots' codes and scales, K and V: [n, 2, H, D]."""
    if codes.dtype == torch.uint8:
        codes = codes.view(torch.float8_e5m2 if fmt == kvq.KVQ_FP8_E5M2 else torch.float8_e4m3fn)
    x = codes.double().cpu().numpy()
    if fmt == kvq.KVQ_INT8_PER_CHANNEL:
        return x * chan
    if scales is None:
        return x
    s = scales.double().cpu().numpy()
    if fmt in kvq.BLOCK_FORMATS:
        return x * s[..., None]
    return x * (s[..., None, None] if s.ndim == 2 else np.repeat(s, group, -1))


def _step(fmt, group, want, slots, bs, chan):
    """Half a step of each stored key element, the most that rounding to a code may be
    off: scale / 2 for integer codes, 2^-4 (e4m3), 2^-3 (e5m2) or 2^-11 (fp16) of the
    value, or half of the type's smallest step."""
    a = np.abs(want)
    if fmt == kvq.KVQ_FP16:
        return a * 2.0 ** -11 + 2.0 ** -25
    if fmt == kvq.KVQ_FP8_E5M2:
        return a * 2.0 ** -3 + 2.0 ** -17
    if fmt == kvq.KVQ_INT8_PER_CHANNEL:
        return np.full_like(a, chan / 2)
    top = 448.0 if fmt in (kvq.KVQ_FP8_E4M3_PER_TOKEN, kvq.KVQ_FP8_E4M3_PER_BLOCK) else \
        7.0 if fmt == kvq.KVQ_INT4_PER_GROUP else 127.0
    if fmt in kvq.BLOCK_FORMATS:
        s = np.zeros_like(a)
        for b in np.unique(slots // bs):
            at = slots // bs == b
            s[at] = a[at].max((0, 2), keepdims=True) / top
    elif fmt in (kvq.KVQ_INT8_PER_TOKEN, kvq.KVQ_FP8_E4M3_PER_TOKEN):
        s = np.broadcast_to(a.max((1, 2), keepdims=True) / top, a.shape)
    else:
        g = a.reshape(*a.shape[:2], -1, group)
        s = np.broadcast_to(g.max(-1, keepdims=True) / top, g.shape).reshape(a.shape)
    return a * 2.0 ** -4 + s * 2.0 ** -10 if top == 448.0 else s / 2


@pytest.mark.parametrize("fmt,group", FORMATS + [(kvq.KVQ_INT8_PER_GROUP, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bs,hq,hkv,d,r,T", [
    (16, 4, 2, 128, 128, 40), (16, 4, 2, 128, 128, 1100), (16, 2, 2, 64, 64, 1300), (32, 2, 1, 128, 96, 1310),
    (64, 2, 2, 128, 128, 70), (64, 4, 2, 128, 128, 1100), (64, 1, 1, 64, 48, 1110), (32, 3, 3, 64, 64, 100),
    (16, 2, 1, 128, 112, 1030), (8, 2, 2, 128, 128, 1100), (16, 2, 2, 128, 16, 1040), (16, 2, 2, 64, 16, 33)])
def test_stored_keys(fmt, group, interleaved, bs, hq, hkv, d, r, T):
    if bs == 8 and fmt == kvq.KVQ_INT4_PER_GROUP:
        pytest.skip("INT4 takes blocks of 16 tokens or more")
    group, norm = min(group, d), bool((T // 10 + interleaved) % 2)
    rng = np.random.default_rng(bs * 1000 + d + r)
    # sequences that begin at block starts and inside blocks, long ones and single tokens
    lens, starts = [], []
    while sum(lens) < T:
        lens.append(int(min(rng.choice([1, 3 * bs, 2 * bs + 5, 300]), T - sum(lens))))
        starts.append(int(rng.choice([0, 0, 3])))
    slots, nb = _slots(rng, lens, bs, starts)
    qkv = _rows(rng, T, hq + 2 * hkv, d, torch.bfloat16 if norm else torch.float16)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    pos = rng.integers(0, 1 << 17, T)
    plan = kvq.kvq_rope_init(r, interleaved)
    w = _t(1 + 0.1 * rng.standard_normal(d).astype(np.float32)) if norm else None
    chan = 0.75  # (absmax 12 * 4 or so without the norm: within 127 steps)
    pool = _plain_pool(fmt, group, nb, bs, hkv, d, torch.full((hkv, d), chan, device=DEV))
    pool.rope_append(plan, q, k, v, _t(pos), _t(slots), q_weight=w, k_weight=w, eps=EPS)
    assert pool.error() == kvq.KVQ_OK
    got = _values(fmt, group, *pool.read_slots(_t(slots)), chan)
    wn = None if w is None else w.cpu().numpy()
    x = k.float().cpu().numpy()
    want = rope(x, pos, frequencies(r), interleaved, 1.0, wn, EPS)
    # in fp32 before the rounding: 2^-19 of the pair, whose ends are at most the head's
    # largest normed element (as in test_rope_append), which moves the scale as well
    reach = np.abs(rope(x, weight=wn, eps=EPS)).max((1, 2), keepdims=True)
    reach = np.broadcast_to(reach.max() if fmt in kvq.BLOCK_FORMATS else reach, want.shape)
    off = np.abs(got[:, 0] - want)
    bound = _step(fmt, group, want, slots, bs, chan) * (1 + 2.0 ** -16) + 2.0 ** -17 * reach
    assert (off <= bound).all(), (off - bound).max()
    # values as they were given
    vw = v.double().cpu().numpy()
    off = np.abs(got[:, 1] - vw)
    assert (off <= _step(fmt, group, vw, slots, bs, chan) * (1 + 2.0 ** -16) + 2.0 ** -20 * np.abs(vw).max()).all()
    pool.close()


@pytest.mark.parametrize("T", [3, 64, 1100])
def test_fp16_blocks_of_64_with_whole_heads_rotated(T):
    """The largest page image beside the largest angle table: 48 KB of shared memory and
    what the kernel has of its own."""
    rng = np.random.default_rng(T)
    d, hkv, bs = 128, 2, 64
    pool = kvq.KVPool(T // bs + 1, bs, hkv, d, kvq.KVQ_FP16, device=DEV)
    x = _rows(rng, T, 2 * hkv, d)
    pos = rng.integers(0, 1 << 17, T)
    slots = np.arange(T)
    pool.rope_append(kvq.kvq_rope_init(d), None, x[:, :hkv], x[:, hkv:], _t(pos), _t(slots))
    assert pool.error() == kvq.KVQ_OK
    k, v = pool.read_values(_t(slots))
    assert torch.equal(v, x[:, hkv:])
    want = rope(x[:, :hkv].float().cpu().numpy(), pos, frequencies(d))
    np.testing.assert_allclose(k.double().cpu().numpy(), want, rtol=2.0 ** -11,
                               atol=2.0 ** -19 * float(x.abs().max()) + 2.0 ** -25)
    pool.close()
