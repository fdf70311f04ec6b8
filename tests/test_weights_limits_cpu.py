"""Sizes whose counts leave 32 bits are refused by kvq_attention_weights before it
could launch (no GPU: a made-up pool and addresses)."""
import pytest

import paged_quantized_kv_kvq_gb300 as kvq
from paged_quantized_kv_kvq_gb300 import build as kbuild
from test_evict_cpu import FakePool, _weights


@pytest.fixture(scope="module", autouse=True)
def L():
    kbuild.build()
    return kvq.lib()


@pytest.mark.parametrize("S", [2 ** 29 - 1, 2 ** 29, 2 ** 30 - 1, 2 ** 30 + 5, 2 ** 31 - 1])
def test_more_sequences_than_shared_memory_holds(L, S):
    """4 bytes of each sequence in shared memory: (S + 1) * 4 passes 2^31 here, and
    2^32, where a sum in 32 bits would look as if it fitted."""
    assert _weights(L, FakePool(hkv=1), S=S, hq=1, mb=2, mc=16, stride=16) == kvq.KVQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("stages_per_row", [107374, 107370])
def test_stages_next_to_32_bits(L, stages_per_row):
    """20000 sequences whose stages of 32 tokens number just under 2^31: shared over the
    warps the count is rounded up, and must not pass 2^31 there."""
    n = 32 * stages_per_row
    assert 2 ** 31 - 2 ** 17 < 20000 * stages_per_row < 2 ** 31
    assert _weights(L, FakePool(hkv=1), S=20000, hq=1, mb=n // 16, mc=n, stride=n) == kvq.KVQ_ERR_UNSUPPORTED
