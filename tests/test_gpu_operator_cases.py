"""The timing cases that append single tokens to blocks with one scale each: every pass
starts from the blocks as they were, so that it rescales what the first one did."""
import importlib.util
import os
import random

import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq

pytestmark = pytest.mark.gpu


def _cases():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")
    spec = importlib.util.spec_from_file_location("operator_cases", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.own = True
    return m


def _single(c):
    return c["op"] == "append" and c["n"] == 1 and "block" in c["fmt"]


def _picked(m):
    rng, out = random.Random(5), [c for c in m.listed() if _single(c)]
    while len(out) < 4:
        out += [c for c in [m.draw(rng)] if _single(c)]
    return out


@pytest.mark.parametrize("i", range(4))
def test_passes_do_the_same_work(i):
    m = _cases()
    c = _picked(m)[i]
    s = m.prepare(c, 11)
    pool = s["pool"]
    g = torch.Generator(device="cuda").manual_seed(1)
    want = None
    for _ in range(3):
        got = {k: v.clone() for k, v in m.run(s).items()}
        want = got if want is None else want
        for k in want:
            assert torch.equal(got[k], want[k]), k
        # scales of the touched blocks, K and V of every head: most of them grow again
        x = 1000 * torch.randn((c["S"], c["hkv"], c["d"]), generator=g, device="cuda").half()
        pool.append(x, x, s["slots"])
    assert pool.error() == kvq.KVQ_OK
