"""Differential attention over every kind of pool against float64."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq
from cache_ops_ref import attention, tokens

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
FORMATS = [(kvq.KVQ_FP4_E2M1, 0), (kvq.KVQ_INT8_PER_BLOCK, 0), (kvq.KVQ_FP8_E4M3_PER_BLOCK, 0), (kvq.KVQ_FP16, 0),
           (kvq.KVQ_INT8_PER_TOKEN, 0), (kvq.KVQ_INT8_PER_CHANNEL, 0), (kvq.KVQ_INT8_PER_GROUP, 64), (kvq.KVQ_INT8_PER_GROUP, 32),
           (kvq.KVQ_FP8_E4M3_PER_TOKEN, 0), (kvq.KVQ_INT4_PER_GROUP, 64), (kvq.KVQ_INT4_PER_GROUP, 16), (kvq.KVQ_FP8_E5M2, 0)]


def _t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _filled(fmt, group, bs, hkv, d, lens, seed=0, fill_byte=0):
    """A pool and its values (float64 [slots, 2, Hkv, D], as the pool itself says what it holds)."""
    rng = np.random.default_rng(seed)
    per = [(n + bs - 1) // bs for n in lens]
    nb = max(sum(per), 1)
    perm, at = rng.permutation(nb), 0
    table = np.zeros((len(lens), max(max(per), 1) + 1), np.int32)
    for s, n in enumerate(per):
        table[s, :n] = perm[at:at + n]
        at += n
    pool = kvq.KVPool(nb, bs, hkv, d, fmt, group, device=DEV, fill_byte=fill_byte)
    slots = np.concatenate([tokens(table, lens, s, bs) for s in range(len(lens))])
    k, v = (rng.standard_normal((len(slots), hkv, d)).astype(np.float16) for _ in range(2))
    chan = None
    if fmt == kvq.KVQ_INT8_PER_CHANNEL:
        kvq.kvq_calibrate_channel_scales(pool.handle, _t(k), _t(v))
        chan = np.stack([np.abs(x.astype(np.float32)).max(0) / np.float32(127) for x in (k, v)]).astype(np.float64)
    vals = np.zeros((nb * bs, 2, hkv, d))
    if len(slots):
        pool.append(_t(k), _t(v), _t(slots))
        codes, scales = pool.read_slots(_t(slots))
        if fmt == kvq.KVQ_FP4_E2M1:
            from fp4_ref import MAGNITUDES
            c = codes.cpu().numpy()
            x = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0)
        else:
            if codes.dtype == torch.uint8:
                codes = codes.view(torch.float8_e5m2 if fmt == kvq.KVQ_FP8_E5M2 else torch.float8_e4m3fn)
            x = codes.double().cpu().numpy()
        if scales is not None:
            s = scales.double().cpu().numpy()
            s = s[..., None] if fmt in kvq.BLOCK_FORMATS else s[..., None, None] if s.ndim == 2 else np.repeat(s, d // s.shape[-1], -1)
            x = x * s
        elif chan is not None:
            x = x * chan
        vals[slots] = x
    return pool, vals, table, np.array(lens, np.int32), rng


def diff_ref(values, q, lens, lam, weight, eps, out_scale, sm_scale=None):
    """float64: values(s) gives sequence s's [L, 2, Hkv, D]; q [S, H, D] single tokens."""
    d = q.shape[-1]
    sm_scale = (d // 2) ** -0.5 if sm_scale is None else sm_scale
    out = []
    for a, b in ((0, d // 2), (d // 2, d)):
        def half(s):
            x = values(s).copy()
            x[:, 0, :, :a] = 0
            x[:, 0, :, b:] = 0
            return x

        out.append(attention(half, q, lens, sm_scale)[0])
    y = out[0] - lam[None, :, None] * out[1]
    if weight is not None:
        den = (y * y).mean(-1, keepdims=True) + eps
        y = np.divide(y, np.sqrt(den), out=np.zeros_like(y), where=den > 0) * weight
    return y * out_scale, out


SUMS = 1e-5        # fp32 sums of a map, of its root mean square
LONG = 3e-4        # where the tensor core's accumulator sums long ranges (formats with scales per token or group)
# prompts: each weight is an fp16 number, within 2^-11 / x of itself, x in [1, 2) its mantissa.  Over mantissas spread
# as logarithms the mean of 1 / x^2 is (1 - 1/4) / (2 ln 2) = 0.54, so the error is 0.73 2^-11 / sqrt(3) in root mean square,
# and a value is a sum of such independent errors: of the map's root mean square that much.  (_near allows ten times it;
# half of it is taken, which holds five of them.)
WEIGHTS = 0.5 * 0.73 * 2.0 ** -11 / 3 ** 0.5


def _near(got, want, maps, lam, weight, out_scale, rel):
    """fp16 results: half a step (2^-11), and the error of the maps, ten times `rel` of their root
    mean square at most, before their difference is taken; the norm multiplies it like the
    value."""
    got = got.astype(np.float64)
    assert np.isfinite(got).all()
    y = maps[0] - lam[None, :, None] * maps[1]
    size = np.sqrt((maps[0] ** 2).mean(-1, keepdims=True)) + np.abs(lam)[None, :, None] * np.sqrt((maps[1] ** 2).mean(-1, keepdims=True))
    gain = np.ones_like(size) * out_scale
    if weight is not None:
        rms = np.sqrt((y ** 2).mean(-1, keepdims=True))
        gain = np.divide(out_scale * np.abs(weight).max(), rms, out=np.zeros_like(rms), where=rms > 0)
    bound = np.abs(want) * 2.0 ** -11 + 10 * rel * size * np.abs(gain) + 2.0 ** -25
    assert (np.abs(got - want) <= bound).all(), np.abs(got - want).max()


SHAPES = [(16, 8, 2, 128, [1, 0, 17, 333, 16, 900]), (32, 4, 1, 64, [31, 33, 500]), (64, 6, 2, 64, [63, 65, 1, 300]),
          (16, 24, 2, 128, [45, 400]), (16, 4, 4, 128, [129, 0, 640]), (32, 5, 1, 128, [70, 2]), (16, 1, 1, 64, [5])]


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("bs,H,hkv,d,lens", SHAPES)
def test_decode(fmt, group, bs, H, hkv, d, lens):
    pool, vals, table, lens, rng = _filled(fmt, group, bs, hkv, d, lens, seed=bs + H, fill_byte=0xFF if fmt == kvq.KVQ_FP4_E2M1 else 0)
    S = len(lens)
    q = rng.standard_normal((S, H, d)).astype(np.float16)
    lam = rng.uniform(-0.5, 1, H).astype(np.float32)
    w = rng.uniform(0.5, 1.5, d).astype(np.float32)
    most = int(max(lens.max(), 1))
    for weight, eps, scale in ((None, 0.0, 1.0), (w, 1e-5, 0.2)):
        want, maps = diff_ref(lambda s: vals[tokens(table, lens, s, bs)], q, lens, lam.astype(np.float64), weight, eps, scale)
        out = pool.diff_decode(_t(q), _t(table), _t(lens), most, _t(lam), None if weight is None else _t(weight), eps, scale)
        assert pool.error() == kvq.KVQ_OK
        _near(out.cpu().numpy(), want, maps, lam, weight, scale, LONG)
        assert (out[_t(lens) == 0] == 0).all()
    pool.close()


@pytest.mark.parametrize("fmt", [kvq.KVQ_INT8_PER_BLOCK, kvq.KVQ_FP16, kvq.KVQ_INT8_PER_TOKEN])
def test_decode_of_eight_token_blocks(fmt):
    pool, vals, table, lens, rng = _filled(fmt, 0, 8, 2, 128, [1, 0, 7, 8, 9, 301], seed=3)
    q, lam = rng.standard_normal((6, 4, 128)).astype(np.float16), np.array([0.3, 0.8, -0.2, 0], np.float32)
    want, maps = diff_ref(lambda s: vals[tokens(table, lens, s, 8)], q, lens, lam.astype(np.float64), None, 0, 1)
    out = pool.diff_decode(_t(q), _t(table), _t(lens), 301, _t(lam))
    _near(out.cpu().numpy(), want, maps, lam, None, 1.0, LONG)
    assert kvq.kvq_diff_prefill_workspace_bytes(pool.handle, 6, 6, 4, 301) == 0
    with pytest.raises(kvq.KVQError) as e:
        kvq.kvq_diff_prefill(pool.handle, _t(q), _t(np.arange(7, dtype=np.int32)), 1, _t(table), _t(lens), 301, 0.125, _t(lam),
                             torch.empty_like(_t(q)), None)
    assert e.value.status == kvq.KVQ_ERR_UNSUPPORTED
    pool.close()


@pytest.mark.parametrize("fmt", [kvq.KVQ_FP4_E2M1, kvq.KVQ_INT8_PER_BLOCK])
def test_decode_precision(fmt):
    """Long sequences split over many warps: fp32 sums within 1e-5 of the maps."""
    pool, vals, table, lens, rng = _filled(fmt, 0, 16, 2, 128, [5000, 9000, 77], seed=9)
    q, lam = rng.standard_normal((3, 4, 128)).astype(np.float16), np.array([0.5, 0.8, 1, 0.2], np.float32)
    w = rng.uniform(0.5, 1.5, 128).astype(np.float32)
    want, maps = diff_ref(lambda s: vals[tokens(table, lens, s, 16)], q, lens, lam.astype(np.float64), w, 1e-5, 0.4)
    out = pool.diff_decode(_t(q), _t(table), _t(lens), 9000, _t(lam), _t(w), 1e-5, 0.4)
    _near(out.cpu().numpy(), want, maps, lam, w, 0.4, SUMS)
    pool.close()


@pytest.mark.parametrize("fmt", [kvq.KVQ_FP4_E2M1, kvq.KVQ_INT8_PER_BLOCK])
@pytest.mark.parametrize("S", [2048, 2049])
def test_decode_of_many_sequences(fmt, S):
    """As many sequences as the merge counts itself, and one more, a few of them cut."""
    lens = np.random.default_rng(S).integers(0, 12, S)
    lens[[0, 700, S - 1]] = 3000, 1777, 2500
    pool, vals, table, lens, rng = _filled(fmt, 0, 16, 1, 64, list(lens), seed=1)
    q = rng.standard_normal((S, 2, 64)).astype(np.float16)
    lam, w = np.array([0.4, 0.7], np.float32), rng.uniform(0.5, 1.5, 64).astype(np.float32)
    out = pool.diff_decode(_t(q), _t(table), _t(lens), 3000, _t(lam), _t(w)).cpu().numpy()
    assert pool.error() == kvq.KVQ_OK
    pick = np.unique(np.concatenate([[0, 1, 699, 700, 701, S - 2, S - 1], rng.integers(0, S, 30)]))
    want, maps = diff_ref(lambda i: vals[tokens(table, lens, pick[i], 16)], q[pick], lens[pick], lam.astype(np.float64), w, 1e-5, 1.0)
    _near(out[pick], want, maps, lam, w, 1.0, SUMS)
    pool.close()


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("bs,H,hkv,d,lens,n", [
    (16, 4, 2, 128, [40, 0, 17, 200], [40, 0, 5, 130]), (32, 3, 1, 64, [150, 64, 1], [1, 64, 1]), (64, 16, 2, 128, [70, 300], [9, 1]),
    (16, 2, 2, 64, [129], [129])])
def test_prefill(fmt, group, bs, H, hkv, d, lens, n):
    pool, vals, table, lens, rng = _filled(fmt, group, bs, hkv, d, lens, seed=bs + H, fill_byte=0xFF if fmt == kvq.KVQ_FP4_E2M1 else 0)
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    T = int(start[-1])
    q = rng.standard_normal((T + 3, H, d)).astype(np.float16)
    lam, w = rng.uniform(-0.5, 1, H).astype(np.float32), rng.uniform(0.5, 1.5, d).astype(np.float32)
    most = int(lens.max())
    rows_lens = np.concatenate([np.arange(lens[s] - n[s], lens[s]) + 1 for s in range(len(n))]).astype(np.int32)
    seq = np.repeat(np.arange(len(n)), n)
    for weight, eps, scale in ((w, 1e-5, 0.2), (None, 0.0, 1.5)):
        want, maps = diff_ref(lambda r: vals[tokens(table[seq], rows_lens, r, bs)], q[:T], rows_lens, lam.astype(np.float64), weight, eps, scale)
        ws = torch.full((kvq.kvq_diff_prefill_workspace_bytes(pool.handle, len(n), T + 3, H, most),), 0xFF, dtype=torch.uint8, device=DEV)
        out = torch.full((T + 3, H, d), 7.0, dtype=torch.float16, device=DEV)
        kvq.kvq_diff_prefill(pool.handle, _t(q), _t(start), max(n), _t(table), _t(lens), most, (d // 2) ** -0.5, _t(lam), out, ws,
                             None if weight is None else _t(weight), eps, scale)
        assert pool.error() == kvq.KVQ_OK
        _near(out[:T].cpu().numpy(), want, maps, lam, weight, scale, LONG)
        assert (out[T:] == 7).all()
    pool.close()


@pytest.mark.parametrize("fmt", [kvq.KVQ_FP4_E2M1, kvq.KVQ_INT8_PER_BLOCK])
@pytest.mark.parametrize("H,hkv,d,L,n", [(16, 4, 128, 1200, 1200), (2, 1, 64, 3000, 700), (8, 8, 128, 513, 512), (12, 2, 64, 260, 259)])
def test_prefill_of_many_tiles(fmt, H, hkv, d, L, n):
    """Several work items per SM, chunks that begin inside a context, heads that share tiles;
    rows drawn from all over."""
    pool, vals, table, lens, rng = _filled(fmt, 0, 16, hkv, d, [L, 40, L // 2], seed=H)
    news = [n, 40, 1]
    start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    T = int(start[-1])
    q = rng.standard_normal((T, H, d)).astype(np.float16)
    lam, w = rng.uniform(0, 1, H).astype(np.float32), rng.uniform(0.5, 1.5, d).astype(np.float32)
    out = pool.diff_prefill(_t(q), _t(start), n, _t(table), _t(lens), L, _t(lam), _t(w), 1e-5, 0.5)
    assert pool.error() == kvq.KVQ_OK
    rows_lens = np.concatenate([np.arange(lens[s] - news[s], lens[s]) + 1 for s in range(3)]).astype(np.int32)
    seq = np.repeat(np.arange(3), news)
    pick = np.unique(np.concatenate([rng.integers(0, T, 40), [0, n - 1, n, T - 2, T - 1], np.arange(n - 9, n)]))
    want, maps = diff_ref(lambda r: vals[tokens(table[seq[pick]], rows_lens[pick], r, 16)], q[pick], rows_lens[pick],
                          lam.astype(np.float64), w, 1e-5, 0.5)
    _near(out.cpu().numpy()[pick], want, maps, lam, w, 0.5, SUMS + WEIGHTS)
    pool.close()


def test_rows_without_tokens_and_zero_rows():
    """A context shorter than its chunk leaves rows with nothing (zeros, flagged); lambda 1
    with equal maps leaves zeros that a norm without eps keeps."""
    pool, vals, table, lens, rng = _filled(kvq.KVQ_FP16, 0, 16, 1, 128, [5, 40])
    q = rng.standard_normal((12, 2, 128)).astype(np.float16)
    start = np.array([0, 9, 12], np.int32)
    lam, w = np.array([0.5, 0.1], np.float32), np.ones(128, np.float32)
    out = pool.diff_prefill(_t(q), _t(start), 9, _t(table), _t(lens), 40, _t(lam), _t(w))
    assert pool.error() == kvq.KVQ_ERR_OUT_OF_RANGE
    assert (out[:4] == 0).all() and torch.isfinite(out).all() and (out[4:] != 0).any(-1).all()
    k = rng.standard_normal((40, 1, 128)).astype(np.float16)
    k[..., 64:] = k[..., :64]
    qq = rng.standard_normal((1, 1, 128)).astype(np.float16)
    qq[..., 64:] = qq[..., :64]
    pool.append(_t(k), _t(k), _t(tokens(table, lens, 1, 16)))
    one = pool.diff_decode(_t(qq), _t(table[1:]), _t(lens[1:]), 40, _t(np.ones(1, np.float32)), _t(w), eps=0.0)
    assert torch.isfinite(one).all()
    pool.close()


def test_refusals():
    pool, vals, table, lens, rng = _filled(kvq.KVQ_FP4_E2M1, 0, 16, 2, 128, [50, 20])
    q, lam, out = _t(rng.standard_normal((2, 4, 128)).astype(np.float16)), torch.zeros(4, device=DEV), torch.empty((2, 4, 128), dtype=torch.float16, device=DEV)
    T, L = _t(table), _t(lens)
    need = kvq.kvq_diff_decode_workspace_bytes(pool.handle, 2, 4, 50)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def status(f, *a, **kw):
        with pytest.raises(kvq.KVQError) as e:
            f(*a, **kw)
        return e.value.status

    f = kvq.kvq_diff_decode
    bad = kvq.KVQ_ERR_INVALID_ARG
    assert status(f, pool.handle, q, T, L, 50, 0.1, lam, out, ws, None, -1.0) == bad
    assert status(f, pool.handle, q, T, L, 50, 0.1, lam, out, ws, None, float("nan")) == bad
    assert status(f, pool.handle, q, T, L, 50, 0.1, lam, out, ws, None, 0.0, float("inf")) == bad
    assert status(f, pool.handle, q, T, L, 50, float("nan"), lam, out, ws) == bad
    assert status(f, pool.handle, q, T, L, 16 * T.shape[1] + 1, 0.1, lam, out, ws) == bad
    assert status(f, pool.handle, q, T, L, 50, 0.1, lam, out, None) == kvq.KVQ_ERR_WORKSPACE
    assert status(f, pool.handle, q, T, L, 50, 0.1, lam, out, ws[:-1]) == kvq.KVQ_ERR_WORKSPACE
    assert status(f, pool.handle, q, T, L, 50, 0.1, lam, out, torch.empty(need + 256, dtype=torch.uint8, device=DEV)[1:]) == bad
    g, qs = kvq.kvq_diff_prefill, _t(np.array([0, 1, 2], np.int32))
    assert status(g, pool.handle, q, qs, 1, T, L, 50, 0.1, lam, out, None) == kvq.KVQ_ERR_WORKSPACE
    assert status(g, pool.handle, q, qs, -1, T, L, 50, 0.1, lam, out, None) == bad
    big = torch.empty(kvq.kvq_diff_prefill_workspace_bytes(pool.handle, 2, 2, 4, 50), dtype=torch.uint8, device=DEV)
    odd = torch.empty(2 * 4 * 128 + 1, dtype=torch.float16, device=DEV)[1:].view(2, 4, 128)
    assert status(g, pool.handle, q, qs, 1, T, L, 50, 0.1, lam, odd, big) == bad
    for name, x in (("lam", lam.double()), ("out", out.float()), ("q", q.float())):
        with pytest.raises(ValueError, match="must be"):
            f(pool.handle, **{**dict(q=q, block_table=T, context_lens=L, max_context_len=50, sm_scale=0.1, lam=lam, out=out, workspace=ws), name: x})
    assert pool.error() == kvq.KVQ_OK
    pool.close()


def test_captured_and_on_another_stream():
    pool, vals, table, lens, rng = _filled(kvq.KVQ_FP4_E2M1, 0, 16, 2, 128, [500, 20])
    q, lam = _t(rng.standard_normal((2, 4, 128)).astype(np.float16)), torch.rand(4, device=DEV)
    T, L, w = _t(table), _t(lens), torch.rand(128, device=DEV)
    want = pool.diff_decode(q, T, L, 500, lam, w)
    qs = _t(np.array([0, 1, 2], np.int32))
    want_p = pool.diff_prefill(q, qs, 1, T, L, 500, lam, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(50_000_000)
    got, got_p = pool.diff_decode(q, T, L, 500, lam, w, stream=side), pool.diff_prefill(q, qs, 1, T, L, 500, lam, w, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(got_p, want_p)
    torch.cuda.synchronize()
    out, out_p = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(max(kvq.kvq_diff_decode_workspace_bytes(pool.handle, 2, 4, 500),
                         kvq.kvq_diff_prefill_workspace_bytes(pool.handle, 2, 2, 4, 500)), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        kvq.kvq_diff_decode(pool.handle, q, T, L, 500, 64 ** -0.5, lam, out, ws, w)
        kvq.kvq_diff_prefill(pool.handle, q, qs, 1, T, L, 500, 64 ** -0.5, lam, out_p, ws, w)
    for _ in range(2):
        out.zero_()
        out_p.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out_p, want_p)
    pool.close()
