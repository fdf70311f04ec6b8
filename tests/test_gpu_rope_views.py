"""Views whose strides along a dimension of one row or one head say nothing: the same
bits as of contiguous rows."""
import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _like(x):
    """x [1, H, D] or [T, 1, D] with another stride along the dimension of one."""
    y = torch.empty((x.shape[1], x.shape[0], x.shape[2]), dtype=x.dtype, device=x.device)
    y = y.copy_(x.transpose(0, 1)).transpose(0, 1)
    assert y.shape == x.shape and y.stride() != x.stride()
    return y


@pytest.mark.parametrize("T,hq,hkv", [(1, 8, 2), (5, 1, 1), (1500, 1, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_strides_of_single_rows_and_heads(T, hq, hkv, d):
    g = torch.Generator(device=DEV).manual_seed(T)
    q, k, v = (torch.randn((T, h, d), generator=g, device=DEV).bfloat16() for h in (hq, hkv, hkv))
    pos = torch.arange(T, device=DEV) * 7
    plan = kvq.kvq_rope_init(d)
    out = [torch.empty(x.shape, dtype=torch.float16, device=DEV) for x in (q, k)]
    kvq.kvq_rope(plan, q, k, pos, *out)
    got = [_like(torch.zeros_like(o)) for o in out]
    kvq.kvq_rope(plan, _like(q), _like(k), pos, *got)
    assert all(torch.equal(a, b) for a, b in zip(out, got))
    pools = [kvq.KVPool(T // 16 + 1, 16, hkv, d, kvq.KVQ_INT8_PER_BLOCK, device=DEV) for _ in range(2)]
    at = torch.arange(T, device=DEV)
    a = pools[0].rope_append(plan, q, k, v, pos, at)
    b = pools[1].rope_append(plan, _like(q), _like(k), _like(v), pos, at)
    assert torch.equal(a, b)
    for x, y in zip(*(p.read_slots(at) for p in pools)):
        assert torch.equal(x, y)
    for p in pools:
        assert p.error() == kvq.KVQ_OK
        p.close()
