"""KVPool's calls on a stream that is not the current one: what they allocate is that
stream's, so neither its filling nor a workspace's next user gets in its way."""
import pytest
import torch

import paged_quantized_kv_kvq_gb300 as kvq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
S, HQ, HKV, D, BS, L = 3, 8, 2, 128, 16, 4000


@pytest.fixture()
def case():
    g = torch.Generator(device=DEV).manual_seed(1)
    nb = -(-L // BS)
    pool = kvq.KVPool(S * nb, BS, HKV, D, kvq.KVQ_INT8_PER_BLOCK, device=DEV)
    n = S * nb * BS
    pool.append(torch.randn((n, HKV, D), generator=g, device=DEV).half(), torch.randn((n, HKV, D), generator=g, device=DEV).half(),
                torch.arange(n, device=DEV))
    q = torch.randn((S, HQ, D), generator=g, device=DEV).half()
    table = torch.arange(S * nb, dtype=torch.int32, device=DEV).view(S, nb)
    lens = torch.full((S,), L, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    yield pool, q, table, lens
    pool.close()


def _side():
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    return side


def _behind(call, raw):
    """call(stream) on a side stream while the current stream has work queued before
    anything that it is given now: the results once both are done."""
    side = _side()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    out = call(side.cuda_stream if raw else side)
    side.synchronize()
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("raw", [False, True])
def test_evicted_scores_are_not_cleared_afterwards(case, raw):
    pool, q, table, lens = case
    w = torch.rand((S, HKV, L), device=DEV)
    want = pool.evict_blocks(w, table, lens, L, 20, 1, 2)
    got = _behind(lambda st: pool.evict_blocks(w, table, lens, L, 20, 1, 2, stream=st), raw)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert got[3].any()


@pytest.mark.parametrize("raw", [False, True])
def test_values_read_on_another_stream(case, raw):
    pool = case[0]
    at = torch.arange(0, 300, 7, device=DEV)
    want = pool.read_values(at)
    got = _behind(lambda st: pool.read_values(at, stream=st), raw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["decode", "decode_lse", "cascade_decode", "decode_step"])
def test_a_workspace_goes_back_to_its_stream(case, name, monkeypatch):
    """Once the call has returned, its workspace must not become the current stream's."""
    pool, q, table, lens = case
    new = torch.zeros((S, HKV, D), dtype=torch.float16, device=DEV)
    seen = []
    raw = "kvq_paged_" + name if name.startswith("decode") and name != "decode_step" else "kvq_" + name
    real = getattr(kvq, raw)

    def spy(*a):
        seen.extend((t.data_ptr(), t.numel()) for t in a if getattr(t, "dtype", None) == torch.uint8)
        return real(*a)

    monkeypatch.setattr(kvq, raw, spy)
    side = _side()
    args = {"decode": (q, table, lens, L), "decode_lse": (q, table, lens, L), "cascade_decode": (q, table, lens, L, 4),
            "decode_step": (new, new, q, table, lens, L)}[name]
    out = getattr(pool, name)(*args, stream=side)
    ptr, n = seen[0]
    mine = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(4)]
    assert ptr not in [t.data_ptr() for t in mine]
    side.synchronize()
    first = out[0] if isinstance(out, tuple) else out
    assert torch.isfinite(first).all()
