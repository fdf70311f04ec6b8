"""Shapes that do not belong to the pool are refused by the bindings of the operators
around the cache (no GPU: host tensors, and a handle that stands for no pool; every
call is refused for its shapes, before its tensors' device is looked at)."""
import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq

BS, HKV, D = 16, 2, 128
HANDLE = kvq.PoolHandle(0)
HANDLE.shape = (BS, HKV, D)


def _half(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def _ints(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


def _refused(match, f, *a, **kw):
    with pytest.raises(ValueError, match=match):
        f(*a, **kw)


@pytest.mark.parametrize("heads,d", [(1, D), (3, D), (HKV, 64)])
@pytest.mark.parametrize("strided", [False, True])
def test_rope_append_rows_of_another_pool(heads, d, strided):
    """A slice of packed rows with fewer heads has a row stride that would do."""
    rows = _half(4, 4 * HKV + heads, d)
    k = rows[:, :heads] if strided else _half(4, heads, d)
    v = rows[:, heads:2 * heads] if strided else _half(4, heads, d)
    _refused("2 kv heads of 128", kvq.kvq_rope_append, HANDLE, None, None, k, v, None, _ints(4, dtype=torch.int64))


@pytest.mark.parametrize("shape", [(5, 1, D), (5, HKV, 64), (5, HKV * D - 8), (4, HKV, D)])
def test_read_values(shape):
    _refused("k_out, v_out must be", kvq.kvq_read_values, HANDLE, _ints(5, dtype=torch.int64), _half(*shape), _half(*shape))


def test_flattened_rows_are_as_good():
    """[n, kv_heads * head_dim] and [num_seqs, num_q_heads * head_dim]: the same memory
    (refused here for being a host's)."""
    _refused("CUDA device", kvq.kvq_read_values, HANDLE, _ints(5, dtype=torch.int64), _half(5, HKV * D), _half(5, HKV * D))
    _refused("CUDA device", kvq.kvq_paged_decode_lse, HANDLE, **_decode(out=torch.zeros((3, 4 * D))))


def _decode(**kw):
    a = dict(q=_half(3, 4, D), block_table=_ints(3, 6), context_lens=_ints(3), max_context_len=96, sm_scale=1.0,
             out=torch.zeros((3, 4, D)), lse=torch.zeros((3, 4)))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,match", [
    (dict(q=_half(3, 4, 64), out=torch.zeros((3, 4, 64))), "head_dim of 128"), (dict(q=_half(3, 3, D), out=torch.zeros((3, 3, D)),
                                                                                lse=torch.zeros((3, 3))), "multiple of its 2"),
    (dict(block_table=_ints(2, 6)), "block_table"), (dict(block_table=_ints(18)), "block_table"),
    (dict(context_lens=_ints(2)), "context_lens"), (dict(out=torch.zeros((3, 4, 64))), "out must"),
    (dict(out=torch.zeros((2, 4, D))), "out must"), (dict(q=_half(12, D)), "q must"), (dict(lse=torch.zeros((2, 4))), "lse must")])
def test_decode_lse(kw, match):
    _refused(match, kvq.kvq_paged_decode_lse, HANDLE, **_decode(**kw))


@pytest.mark.parametrize("kw,match", [
    (dict(q=_half(3, 4, 64)), "head_dim of 128"), (dict(block_table=_ints(2, 6)), "block_table"),
    (dict(context_lens=_ints(4)), "context_lens"), (dict(scores=torch.zeros((3, 1, 96))), "2 kv heads"),
    (dict(scores=torch.zeros((3, 4, 96))), "2 kv heads")])
def test_attention_weights(kw, match):
    a = _decode(scores=torch.zeros((3, HKV, 96)), **kw) if "scores" not in kw else _decode(**kw)
    del a["out"]
    _refused(match, kvq.kvq_attention_weights, HANDLE, **a)


@pytest.mark.parametrize("heads", [1, 3])
def test_evict(heads):
    w = torch.zeros((3, heads, 96))
    _refused("2 kv heads", kvq.kvq_evict_blocks, HANDLE, w, _ints(3, 6), _ints(3), 96, 2, 0, 1, _ints(3, 6), _ints(3))


def test_pool_methods_pass_the_handle_on():
    """KVPool's calls go through the same checks."""

    class Pool(kvq.KVPool):
        def __init__(self):
            self.handle, self.kv_heads, self.head_dim, self.block_size, self.num_blocks = HANDLE, HKV, D, BS, 4
            self.dtype, self.group = kvq.KVQ_FP16, 0

        def close(self):
            pass

    p = Pool()
    k = _half(4, 1, D)
    _refused("2 kv heads of 128", p.rope_append, None, None, k, k, None, _ints(4, dtype=torch.int64))
    _refused("block_table", p.decode_lse, _half(3, 4, D), _ints(2, 6), _ints(3), 96)


def test_a_handle_carries_its_shape(monkeypatch):
    """kvq_alloc_pool notes the shape that it was asked for."""

    class Lib:
        def kvq_alloc_pool(self, *a):
            return kvq.KVQ_OK

    monkeypatch.setattr(kvq, "lib", lambda: Lib())
    assert kvq.kvq_alloc_pool(7, 32, 5, 64, kvq.KVQ_FP16).shape == (32, 5, 64)


def test_read_values_leaves_no_row_undefined(monkeypatch):
    """Rows of padding and of slots outside the pool, which the library does not write."""
    pool = kvq.KVPool.__new__(kvq.KVPool)
    pool.handle, pool.kv_heads, pool.head_dim = HANDLE, HKV, D
    monkeypatch.setattr(kvq, "kvq_read_values", lambda *a: None)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: torch.full(*a, float("nan"), **kw))
    monkeypatch.setattr(torch, "empty_like", lambda t: torch.full(t.shape, float("nan"), dtype=t.dtype))
    k, v = kvq.KVPool.read_values(pool, _ints(3, dtype=torch.int64))
    pool.handle = None
    assert k.shape == v.shape == (3, HKV, D) and (k == 0).all() and (v == 0).all()
