"""Plain references of the operators around the cache, for the tests: numpy, one
definition after the other, no code of the package.  Rotations, norms and
attention are float64; the block quantizer is the format's own fp32 arithmetic,
so that its codes and scales can be compared bit by bit."""
from __future__ import annotations

import math

import numpy as np
import torch

INT8_PER_BLOCK = 7
FP8_E4M3_PER_BLOCK = 8


# ------------------------------------------------------------------ rotation
def frequencies(r, base=10000.0, scaling=0, factor=1.0, orig_len=0.0, low=0.0, high=0.0):
    """Radians per position of the r/2 pairs (scaling: 0 none, 1 linear, 2 stretched
    base, 3 by parts, 4 by bands)."""
    out = []
    if scaling == 2:
        base = base * factor ** (r / (r - 2))
    if scaling == 3:
        lo = max(math.floor(r * math.log(orig_len / (2 * math.pi * high)) / (2 * math.log(base))), 0)
        hi = min(math.ceil(r * math.log(orig_len / (2 * math.pi * low)) / (2 * math.log(base))), r - 1)
    for i in range(r // 2):
        f = base ** (-2 * i / r)
        if scaling == 1:
            f /= factor
        elif scaling == 3:
            t = min(max((i - lo) / ((hi - lo) if hi != lo else 0.001), 0), 1)
            f = t * f / factor + (1 - t) * f
        elif scaling == 4:
            turns = orig_len * f / (2 * math.pi)
            t = min(max((turns - low) / (high - low), 0), 1)
            f = (1 - t) * f / factor + t * f
        out.append(f)
    return np.array(out)


def fractions(freq):
    """Turns per position as the integers a 64-bit fraction holds."""
    return [int(math.ldexp(f / (2 * math.pi), 64)) for f in freq]


def angles(freq, positions):
    """pos * f modulo a turn, by exact integer arithmetic: [T, pairs] in radians."""
    out = np.empty((len(positions), len(freq)))
    for j, f in enumerate(fractions(freq)):
        for t, p in enumerate(positions):
            x = int(p) * f % (1 << 64)
            out[t, j] = (x - (1 << 64) if x >= 1 << 63 else x) * 2.0 ** -64 * 2 * math.pi
    return out


def rope(x, positions=None, freq=None, interleaved=False, magnitude=1.0, weight=None, eps=0.0):
    """x [T, H, D] -> float64 rows after the norm (weight given) and the rotation (freq given)."""
    y = np.array(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if freq is None:
        return y
    r = 2 * len(freq)
    a = angles(freq, positions)[:, None, :]
    c, s = np.cos(a) * magnitude, np.sin(a) * magnitude
    lo, hi = (np.s_[..., 0:r:2], np.s_[..., 1:r:2]) if interleaved else (np.s_[..., :r // 2], np.s_[..., r // 2:r])
    u, v = y[lo].copy(), y[hi].copy()
    y[lo], y[hi] = u * c - v * s, u * s + v * c
    return y


def rope_bound(y, x_normed, r, interleaved, magnitude):
    """Largest error of an fp16 result y of rotating x_normed in fp32: half an fp16
    step of the value, and of each pair 2^-20 from cosine and sine and 2^-21 from
    the norm and the fp32 products, times the pair's length."""
    pair = np.zeros_like(y)
    if r:
        lo, hi = (np.s_[..., 0:r:2], np.s_[..., 1:r:2]) if interleaved else (np.s_[..., :r // 2], np.s_[..., r // 2:r])
        n = magnitude * (np.abs(x_normed[lo]) + np.abs(x_normed[hi]))
        pair[lo], pair[hi] = n, n
    pair[..., r:] = np.abs(x_normed[..., r:])
    return np.abs(y) * 2.0 ** -11 + pair * (2.0 ** -20 + 2.0 ** -21) + 2.0 ** -25


# ------------------------------------------------------------------ one scale per block
def e4m3(x):
    """Nearest e4m3 code bytes of fp32 x, saturating (torch's CPU cast)."""
    t = torch.from_numpy(np.clip(np.asarray(x, np.float32), -448, 448))
    return t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def e4m3_value(c):
    return torch.from_numpy(np.ascontiguousarray(c)).view(torch.float8_e4m3fn).float().numpy()


class BlockCache:
    """Codes [slots, 2, Hkv, D] and scales [blocks, 2, Hkv] of a per-block format."""

    def __init__(self, fmt, num_blocks, bs, hkv, d, sentinel=0):
        self.fmt, self.bs, self.hkv, self.d = fmt, bs, hkv, d
        self.fp8 = fmt == FP8_E4M3_PER_BLOCK
        self.codes = np.full((num_blocks * bs, 2, hkv, d), sentinel,
                             np.uint8 if self.fp8 else np.int8)
        self.scales = np.zeros((num_blocks, 2, hkv), np.float32)

    def _codes(self, x, s):
        s = np.broadcast_to(s, x.shape)
        y = np.divide(x, s, out=np.zeros_like(x), where=s != 0).astype(np.float32)
        if self.fp8:
            return e4m3(y)
        return np.clip(np.rint(y), -127, 127).astype(np.int8)

    def _value(self, c):
        return e4m3_value(c) if self.fp8 else c.astype(np.float32)

    def append(self, k, v, slots):
        """k, v [T, Hkv, D] (fp16 or fp32 values), the tokens of a block side by side."""
        slots = np.asarray(slots)
        top = np.float32(448 if self.fp8 else 127)
        i = 0
        while i < len(slots):
            if slots[i] < 0 or slots[i] >= len(self.codes):
                i += 1
                continue
            b = slots[i] // self.bs
            e = i
            while e < len(slots) and slots[e] >= 0 and slots[e] // self.bs == b:
                e += 1
            at = slots[i:e]
            fresh = (at % self.bs == 0).any()
            others = np.setdiff1d(np.arange(b * self.bs, (b + 1) * self.bs), at)
            for kv, x in enumerate((k, v)):
                for h in range(self.hkv):
                    new = np.asarray(x[i:e, h], np.float32)
                    old = np.float32(0) if fresh else self.scales[b, kv, h]
                    s = max(old, np.float32(np.abs(new).max()) / top)
                    kept = self.codes[others, kv, h]
                    if fresh:
                        kept = np.zeros_like(kept)
                    elif s > old:
                        kept = self._codes((self._value(kept) * old).astype(np.float32), s)
                    self.codes[others, kv, h] = kept
                    self.codes[at, kv, h] = self._codes(new, s)
                    self.scales[b, kv, h] = s
            i = e

    def values(self, slots):
        """float64 values [n, 2, Hkv, D]."""
        slots = np.asarray(slots)
        return self._value(self.codes[slots]).astype(np.float64) * \
            self.scales[slots // self.bs].astype(np.float64)[..., None]

    def decode(self, q, table, lens, sm_scale=None):
        return attention(lambda s: self.values(tokens(table, lens, s, self.bs)), q, lens, sm_scale)[0]


def tokens(table, lens, s, bs):
    """Slots of sequence s's tokens, in order."""
    t = np.arange(int(lens[s]))
    return np.asarray(table)[s, t // bs].astype(np.int64) * bs + t % bs


def attention(values, q, lens, sm_scale=None):
    """float64 attention of single tokens: values(s) gives sequence s's [L, 2, Hkv, D].
    Returns out [S, Hq, D], lse [S, Hq] and each sequence's weights [Hkv, group, L]."""
    q = np.asarray(q, np.float64)
    S, hq, d = q.shape
    sm_scale = d ** -0.5 if sm_scale is None else sm_scale
    out, lse, weights = np.zeros((S, hq, d)), np.full((S, hq), -np.inf), []
    for s in range(S):
        if lens[s] == 0:
            weights.append(None)
            continue
        kv = values(s)
        hkv = kv.shape[2]
        qs = q[s].reshape(hkv, hq // hkv, d)
        z = np.einsum("hgd,thd->hgt", qs, kv[:, 0]) * sm_scale
        m = z.max(-1, keepdims=True)
        p = np.exp(z - m)
        n = p.sum(-1, keepdims=True)
        weights.append(p / n)
        out[s] = np.einsum("hgt,thd->hgd", p / n, kv[:, 1]).reshape(hq, d)
        lse[s] = (m + np.log(n)).reshape(hq)
    return out, lse, weights
