"""Cosines and sines themselves, seen through the fp32 scales of stored keys: with one
channel of a pair at 1 and the rest of its group at 0, the scales of the groups that
the pair's two channels lie in are |cos| / 127 and |sin| / 127."""
import math

import numpy as np
import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq
from test_rope_precision_cpu import KW, exact_angle, exact_turns

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
D, G = 128, 16


@pytest.mark.parametrize("scaling,kw", KW)
def test_cosines_and_sines(scaling, kw):
    """Within 2^-22 up to position 2^26, by angles of 60 digits."""
    rng = np.random.default_rng(scaling)
    pos = np.unique(np.concatenate([[0, 1, 2, 4095, 131071, 1 << 20, (1 << 26) - 1, 1 << 26, -1, -(1 << 26)],
                                    rng.integers(-(1 << 26), 1 << 26, 30), rng.integers(0, 1 << 17, 23)]))
    turns = exact_turns(D, 10000.0, scaling, **kw)
    plan = kvq.kvq_rope_init(D, scaling=scaling, **kw)
    # token (position p, offset o): channel o of groups 0 .. 3 is 1, that is pairs 16 g + o
    T = len(pos) * G
    k = torch.zeros((T, 1, D), dtype=torch.float16, device=DEV)
    at = torch.arange(T, device=DEV)
    for g in range(4):
        k[at, 0, G * g + at % G] = 1
    p = torch.from_numpy(np.repeat(pos, G)).to(DEV)
    pool = kvq.KVPool(-(-T // 16), 16, 1, D, kvq.KVQ_INT8_PER_GROUP, G, device=DEV)
    pool.rope_append(plan, None, k, k, p, at)
    scales = pool.read_slots(at)[1][:, 0, 0].double().cpu().numpy() * 127 / plan.magnitude
    worst = 0.0
    for i, x in enumerate(pos):
        for j in range(D // 2):
            a = exact_angle(turns[j], x)
            got = scales[i * G + j % G, [j // G, 4 + j // G]]
            worst = max(worst, abs(got[0] - abs(math.cos(a))), abs(got[1] - abs(math.sin(a))))
    # (the magnitude, the absmax over 127 and its read-back round fp32 values of at most 1)
    assert worst <= 2.0 ** -22 + 3 * 2.0 ** -24, worst * 2 ** 22
    pool.close()


def test_angles_all_round_the_circle():
    """Within 2^-23 (quarter turns and Taylor series in fp32) of 256000 angles at
    positions up to 2^20, where the fractions are off by no more than 2^-29; the
    scales' division by 127 rounds to 2^-24."""
    rng = np.random.default_rng(8)
    pos = rng.integers(0, 1 << 20, 4000)
    turns = [int(t * 2 ** 96) for t in exact_turns(D, 10000.0)]
    plan = kvq.kvq_rope_init(D)
    T = len(pos) * G
    k = torch.zeros((T, 1, D), dtype=torch.float16, device=DEV)
    at = torch.arange(T, device=DEV)
    for g in range(4):
        k[at, 0, G * g + at % G] = 1
    p = torch.from_numpy(np.repeat(pos, G)).to(DEV)
    pool = kvq.KVPool(-(-T // 16), 16, 1, D, kvq.KVQ_INT8_PER_GROUP, G, device=DEV)
    pool.rope_append(plan, None, k, k, p, at)
    # [position, offset, group] -> [position, pair] of cosines and of sines
    scales = pool.read_slots(at)[1][:, 0, 0].double().cpu().numpy().reshape(len(pos), G, 8) * 127
    cos, sin = (scales[:, :, 4 * i:4 * i + 4].transpose(0, 2, 1).reshape(len(pos), D // 2) for i in (0, 1))
    a = np.array([[t * int(x) % (1 << 96) for t in turns] for x in pos], dtype=np.float64) * (2 * math.pi / 2.0 ** 96)
    worst = max(np.abs(cos - np.abs(np.cos(a))).max(), np.abs(sin - np.abs(np.sin(a))).max())
    assert worst <= 2.0 ** -23 + 2.0 ** -24 + 2.0 ** -29, worst * 2 ** 23
    pool.close()
