"""Differential attention whose maps all but cancel: the weights of the maps reach the values
with their full precision, whatever the pool's format and the entry point."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq
from cache_ops_ref import tokens
from test_gpu_diff import FORMATS, _filled, _t, diff_ref

pytestmark = pytest.mark.gpu

# Error of a map, in its root mean square, at up to 320 keys: 40 sums of the tensor core (16 keys
# each, high and low parts), every one within 2^-23 of itself (truncated), 4.8e-6; as much again for
# what a product's 16 terms lose beside the largest; fp32 sums of the weights, 90 of 2^-24 at worst,
# 5.4e-6; two fp16 parts of a weight, 2^-22.  Scores of up to 16 in magnitude, whose four sums lose
# 2^-23 each of partial sums of twice that, put a weight off by 1.5e-5 of itself, which moves a map by
# that much of the difference between values, a third of them here: 5e-6.  Together 2.1e-5.
FINE = 2.0 ** -15


def _close(got, want, maps, lam, weight, eps, out_scale):
    """Half an fp16 step, and FINE of the maps' root mean squares.  The norm y -> f y, f = 1 / sqrt(mean(y^2) + eps),
    makes of an error e of y at most f e and, from the change of f, f^3 |y| mean(|y e|) <= f e again; f is
    1 / sqrt(eps) where the maps are equal (a row with one key and lambda 1)."""
    got = got.astype(np.float64)
    assert np.isfinite(got).all()
    y = maps[0] - lam[None, :, None] * maps[1]
    rms = [np.sqrt((x ** 2).mean(-1, keepdims=True)) for x in (*maps, y)]
    size = rms[0] + np.abs(lam)[None, :, None] * rms[1]
    gain = out_scale * np.ones_like(size)
    if weight is not None:
        gain = 2 * out_scale * np.abs(weight).max() / np.sqrt(rms[2] ** 2 + eps)
    bound = np.abs(want) * 2.0 ** -11 + FINE * size * gain + 2.0 ** -25
    assert (np.abs(got - want) <= bound).all(), (np.abs(got - want) / bound).max()


def _put(pool, fmt, slots, k, v):
    """Stores rows and returns what the pool then holds, float64 [n, 2, Hkv, D]."""
    if fmt == kvq.KVQ_INT8_PER_CHANNEL:
        kvq.kvq_calibrate_channel_scales(pool.handle, _t(k), _t(v))
    pool.append(_t(k), _t(v), _t(slots))
    codes, scales = pool.read_slots(_t(slots))
    d = k.shape[-1]
    if fmt == kvq.KVQ_FP4_E2M1:
        from fp4_ref import MAGNITUDES
        c = codes.cpu().numpy()
        x = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0)
    else:
        if codes.dtype == torch.uint8:
            codes = codes.view(torch.float8_e5m2 if fmt == kvq.KVQ_FP8_E5M2 else torch.float8_e4m3fn)
        x = codes.double().cpu().numpy()
    if fmt == kvq.KVQ_INT8_PER_CHANNEL:
        return x * np.stack([np.abs(r.astype(np.float32)).max(0) / np.float32(127) for r in (k, v)]).astype(np.float64)
    if scales is None:
        return x
    s = scales.double().cpu().numpy()
    return x * (s[..., None] if fmt in kvq.BLOCK_FORMATS else s[..., None, None] if s.ndim == 2 else np.repeat(s, d // s.shape[-1], -1))


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
def test_maps_that_cancel(fmt, group, d):
    """Equal keys but for one token of the first map, values around a mean per channel, lambda 1
    and close to it: the equal weights are rounded alike, so that what they lose does not
    average out, and the difference is a small part of the maps."""
    if group > d:
        pytest.skip("a group has more channels than a head")
    bs, L, H, hkv = 16, 300, 4, 2
    pool, _, table, lens, rng = _filled(fmt, group, bs, hkv, d, [L, 77], seed=d)
    slots = np.concatenate([tokens(table, lens, s, bs) for s in range(2)])
    k = np.repeat(rng.standard_normal((1, hkv, d)), len(slots), 0)
    k[[0, L], :, :d // 2] *= 1.7
    v = (rng.choice([-1.0, 1.0], (1, hkv, d)) * rng.uniform(4, 8, (1, hkv, d))) * (1 + 0.3 * rng.standard_normal((len(slots), hkv, d)))
    vals = np.zeros((int(slots.max()) + 1, 2, hkv, d))
    vals[slots] = _put(pool, fmt, slots, k.astype(np.float16), v.astype(np.float16))
    start = np.array([0, L, L + 77], np.int32)
    q = rng.standard_normal((L + 77, H, d)).astype(np.float16)
    lam = np.array([1.0, 0.98, 1.0, 0.9], np.float32)
    w = rng.uniform(0.5, 1.5, d).astype(np.float32)
    rows_lens = np.concatenate([np.arange(n) + 1 for n in (L, 77)]).astype(np.int32)
    seq = np.repeat([0, 1], [L, 77])
    pick = np.concatenate([np.arange(0, L, 7), [62, 63, 64, 65, L - 1], np.arange(L, L + 77, 5), [L + 76]])
    last = np.array([L - 1, L + 76])
    for weight, eps, scale in ((None, 0.0, 1.0), (w, 1e-5, 0.2)):
        def ref(rows):
            return diff_ref(lambda r: vals[tokens(table[seq[rows]], rows_lens[rows], r, bs)], q[rows], rows_lens[rows], lam.astype(np.float64),
                            weight, eps, scale)

        wt = None if weight is None else _t(weight)
        out = pool.diff_prefill(_t(q), _t(start), L, _t(table), _t(lens), L, _t(lam), wt, eps, scale).cpu().numpy()
        one = pool.diff_decode(_t(q[last]), _t(table), _t(lens), L, _t(lam), wt, eps, scale).cpu().numpy()
        assert pool.error() == kvq.KVQ_OK
        _close(one, *ref(last), lam, weight, eps, scale)
        _close(out[pick], *ref(pick), lam, weight, eps, scale)
    pool.close()


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("bs,H,hkv,d,lens,n", [(16, 4, 2, 128, [40, 0, 17, 300], [40, 0, 5, 130]), (32, 6, 2, 64, [150, 64, 1], [1, 64, 1])])
def test_short_contexts_in_every_format(fmt, group, bs, H, hkv, d, lens, n):
    """Random rows, single tokens and prompts, held to the same bound in every format."""
    pool, vals, table, lens, rng = _filled(fmt, group, bs, hkv, d, lens, seed=bs + H)
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    T = int(start[-1])
    q = rng.standard_normal((T, H, d)).astype(np.float16)
    lam, w = rng.uniform(-0.5, 1, H).astype(np.float32), rng.uniform(0.5, 1.5, d).astype(np.float32)
    most = int(lens.max())
    rows_lens = np.concatenate([np.arange(lens[s] - n[s], lens[s]) + 1 for s in range(len(n))]).astype(np.int32)
    seq = np.repeat(np.arange(len(n)), n)
    want, maps = diff_ref(lambda r: vals[tokens(table[seq], rows_lens, r, bs)], q, rows_lens, lam.astype(np.float64), w, 1e-5, 0.2)
    out = pool.diff_prefill(_t(q), _t(start), max(n), _t(table), _t(lens), most, _t(lam), _t(w), 1e-5, 0.2)
    _close(out.cpu().numpy(), want, maps, lam, w, 1e-5, 0.2)
    qs = rng.standard_normal((len(n), H, d)).astype(np.float16)
    want, maps = diff_ref(lambda s: vals[tokens(table, lens, s, bs)], qs, lens, lam.astype(np.float64), w, 1e-5, 0.2)
    out = pool.diff_decode(_t(qs), _t(table), _t(lens), most, _t(lam), _t(w), 1e-5, 0.2)
    _close(out.cpu().numpy(), want, maps, lam, w, 1e-5, 0.2)
    assert pool.error() == kvq.KVQ_OK
    pool.close()
