"""Plain reference of the cache in 4-bit floats, for the tests: numpy, the nearest value
of a table by search, no code of the package.  Quotients are fp32, as the format has
them; everything else is exact."""
from __future__ import annotations

import numpy as np

from cache_ops_ref import attention, tokens

GROUP = 16
MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
# scale bytes 0 .. 0xE2 (10240): 5 exponent bits (bias 15), 3 of mantissa, subnormals
SCALES = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 15)
                   for e in range(31) for m in range(8)])
SCALES = SCALES[SCALES <= 10240]


def nearest(x, table):
    """Index of the value of the ascending table nearest to each x >= 0 (even index at a
    tie, the last one beyond the table; NaN: the last one)."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    with np.errstate(invalid="ignore"):
        up, down = table[hi] - x, x - table[lo]
        i = np.where(up < down, hi, np.where(up > down, lo, np.where(hi % 2 == 0, hi, lo)))
    return np.where(np.isnan(x) | (x >= table[-1]), len(table) - 1, i)


def quantize(x):
    """(codes uint8 like x, scale bytes uint8 [..., D/16]) of fp32-valued rows x [..., D]."""
    x = np.asarray(x, np.float32)
    y = x.reshape(*x.shape[:-1], -1, GROUP)
    amax = np.fmax.reduce(np.abs(y), -1)
    amax = np.where(np.isnan(amax), np.float32(0), amax)  # a group of nothing but NaN
    sb = nearest(amax / np.float32(6), SCALES).astype(np.uint8)
    s = SCALES[sb].astype(np.float32)[..., None]
    with np.errstate(invalid="ignore", over="ignore"):
        q = np.divide(y, s, out=np.zeros_like(y), where=s != 0)
    mag = nearest(np.abs(q), MAGNITUDES)
    code = mag + 8 * (np.signbit(q) & ~np.isnan(q))
    code = np.where(s == 0, 0, code)
    return code.reshape(x.shape).astype(np.uint8), sb


def values(codes, scale_bytes):
    """float64 values of codes [..., D] at scale bytes [..., D/16]."""
    m = MAGNITUDES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return (m.reshape(*m.shape[:-1], -1, GROUP) * SCALES[scale_bytes][..., None]).reshape(m.shape)


class Fp4Cache:
    """Codes [slots, 2, Hkv, D] and scale bytes [slots, 2, Hkv, D/16]."""

    def __init__(self, num_blocks, bs, hkv, d):
        self.bs, self.hkv, self.d, self.blocks = bs, hkv, d, num_blocks
        self.codes = np.zeros((num_blocks * bs, 2, hkv, d), np.uint8)
        self.scales = np.zeros((num_blocks * bs, 2, hkv, d // GROUP), np.uint8)

    def append(self, k, v, slots):
        slots = np.asarray(slots)
        ok = (slots >= 0) & (slots < len(self.codes))
        for kv, x in enumerate((k, v)):
            c, s = quantize(np.asarray(x, np.float32)[ok])
            self.codes[slots[ok], kv] = c
            self.scales[slots[ok], kv] = s

    def values(self, slots):
        return values(self.codes[slots], self.scales[slots])

    def attend(self, q, table, lens, sm_scale=None):
        return attention(lambda s: self.values(tokens(table, lens, s, self.bs)), q, lens, sm_scale)

    def decode(self, q, table, lens, sm_scale=None):
        return self.attend(q, table, lens, sm_scale)[0]
