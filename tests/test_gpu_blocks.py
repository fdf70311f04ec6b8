"""A step's block tables, slot map and positions against a plain walk over the sequences."""
import numpy as np
import pytest
import torch

import blocks_ref
import paged_quantized_kv_kvq_gb300 as kvq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
I32, I64 = torch.int32, torch.int64


def _t(x, dtype=I32):
    return torch.tensor(np.asarray(x), dtype=dtype, device=DEV)


def _pool(nb, bs):
    return kvq.KVPool(nb, bs, 1, 64, kvq.KVQ_FP8_E5M2, device=DEV)


def _extend(pool, n, table, lens, free, count, max_tokens, in_place=False):
    t, L, f, c = _t(table), _t(lens), _t(free), _t([count])
    lo, co = (L, c) if in_place else (torch.full_like(L, -99), torch.full_like(c, -99))
    q = torch.full((len(lens) + 1,), -99, dtype=I32, device=DEV)
    s, p = (torch.full((max_tokens,), -99, dtype=I64, device=DEV) for _ in range(2))
    kvq.kvq_extend_tables(pool.handle, _t(n), t, L, f, c, lo, co, q, s, p)
    assert torch.equal(f, _t(free))
    return {"table": t, "lens": lo, "count": co, "q_start": q, "slots": s, "positions": p}


def _same(got, want):
    for k, w in want.items():
        np.testing.assert_array_equal(got[k].cpu().numpy().reshape(np.shape(w)), w, err_msg=k)


def _case(rng, S, bs, most, new, spare):
    lens = rng.integers(0, most + 1, S) * (rng.random(S) < 0.9)
    n = rng.integers(0, new + 1, S) * (rng.random(S) < 0.8)
    held, end = -(-lens // bs), -(-(lens + n) // bs)
    width = int(max(end.max(initial=1), 1)) + 1
    total = int(end.sum()) + spare
    ids = rng.permutation(total)
    table = np.full((S, width), -7, np.int32)
    at = 0
    for s in range(S):
        table[s, :held[s]] = ids[at:at + held[s]]
        at += held[s]
    free = np.full(total + 3, -1, np.int32)
    free[:total - at] = ids[at:]
    return lens.astype(np.int32), n.astype(np.int32), table, free, total - at, total


@pytest.mark.parametrize("S,bs,most,new,spare,pad", [
    (1, 16, 100, 40, 0, 0), (1, 16, 0, 1, 0, 5), (3, 8, 30, 20, 4, 7), (64, 16, 2000, 1, 10, 0), (64, 32, 500, 300, 3, 100),
    (511, 16, 60, 5, 2, 1), (512, 64, 300, 9, 0, 0), (513, 16, 100, 17, 9, 33), (2000, 16, 90, 3, 5, 0), (16384, 16, 20, 2, 5, 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_extend(S, bs, most, new, spare, pad, in_place):
    rng = np.random.default_rng(S + bs)
    lens, n, table, free, count, total = _case(rng, S, bs, most, new, spare)
    pool = _pool(max(total, 1), bs)
    rows = int(n.sum()) + pad
    want, err = blocks_ref.extend(n, table, lens, free, count, bs, total, rows)
    assert not err
    _same(_extend(pool, n, table, lens, free, count, rows, in_place), want)
    assert pool.error() == kvq.KVQ_OK
    pool.close()


@pytest.mark.parametrize("S", [5, 700])
@pytest.mark.parametrize("trouble", ["blocks", "rows", "row", "negative", "ids", "count", "far"])
def test_sequences_that_are_not_served(S, trouble):
    """Too few free blocks, rows or table entries, negative numbers, ids outside the pool, a
    count outside the list, lengths next to 2^31: flagged, the others served."""
    rng = np.random.default_rng(S)
    bs = 16
    lens, n, table, free, count, total = _case(rng, S, bs, 100, 60, 0)
    rows = int(n.sum())
    if trouble == "blocks":
        count //= 2
    elif trouble == "rows":
        rows //= 2
    elif trouble == "row":
        n[S // 2] = 16 * table.shape[1] + 1 - lens[S // 2]
        rows = int(n.sum())
    elif trouble == "negative":
        n[1], lens[S // 2], lens[S - 1], n[S - 1] = -5, -3, -1, -1
        rows = int(np.maximum(n, 0).sum())
    elif trouble == "ids":
        free[count - 1], free[0] = total + 5, -2
        s = int(np.argmax((lens % bs != 0) & (n > 0)))
        table[s, lens[s] // bs] = 1 << 30
    elif trouble == "count":
        count = len(free) + 7
    else:
        n[0], lens[1] = 2 ** 31 - 1, 2 ** 31 - 1
        n[S - 1] = 2 ** 31 - 1
    pool = _pool(total, bs)
    want, err = blocks_ref.extend(n if trouble != "far" else np.where(n > 1 << 30, rows + 1, n), table, lens, free, count, bs, total, rows)
    assert err
    got = _extend(pool, n, table, lens, free, count, rows)
    if trouble == "far":  # (positions of rows that nobody is served)
        del want["positions"]
    _same(got, want)
    assert pool.error() == kvq.KVQ_ERR_OUT_OF_RANGE
    pool.close()


def test_extend_of_nothing():
    """No sequence, no row, an empty list."""
    pool = _pool(4, 16)
    q, c = torch.full((1,), 9, dtype=I32, device=DEV), _t([2])
    s, p = torch.full((70,), 9, dtype=I64, device=DEV), torch.full((70,), 9, dtype=I64, device=DEV)
    none = torch.empty(0, dtype=I32, device=DEV)
    kvq.kvq_extend_tables(pool.handle, none, torch.empty((0, 3), dtype=I32, device=DEV), none, _t([3, 1, 0]), c, none, c, q, s, p)
    assert q.item() == 0 and c.item() == 2 and (s == -1).all() and (p == 0).all()
    z = torch.empty(0, dtype=I64, device=DEV)
    lens, q2 = _t([5, 0]), torch.full((3,), 9, dtype=I32, device=DEV)
    c0 = _t([0])
    kvq.kvq_extend_tables(pool.handle, _t([0, 0]), _t([[1, 2], [0, 0]]), lens, none, c0, lens, c0, q2, z, z)
    assert lens.tolist() == [5, 0] and q2.tolist() == [0, 0, 0] and c0.item() == 0
    assert pool.error() == kvq.KVQ_OK
    pool.close()


@pytest.mark.parametrize("S,bs,most,shared", [(1, 16, 40, 0), (7, 8, 100, 1), (64, 16, 3000, 0), (300, 32, 2000, 2), (513, 16, 40, 0),
                                              (4, 16, 100000, 3), (3000, 16, 30, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_release(S, bs, most, shared, in_place):
    rng = np.random.default_rng(S)
    old = rng.integers(0, most + 1, S)
    new = np.where(rng.random(S) < 0.4, 0, rng.integers(0, most + 1, S))
    held = -(-old // bs)
    total = int(held.sum()) + 5
    ids = rng.permutation(total).astype(np.int32)
    table = np.full((S, int(held.max()) + 1), -1, np.int32)
    at = 0
    for s in range(S):
        table[s, :held[s]] = ids[at:at + held[s]]
        at += held[s]
    free = np.full(total, -1, np.int32)
    free[:3] = ids[at:at + 3]
    pool = _pool(total, bs)
    want, count, err = blocks_ref.release(table, old, new, free, 3, bs, total, shared)
    assert not err
    f, c = _t(free), _t([3])
    co = c if in_place else _t([-9])
    kvq.kvq_release_blocks(pool.handle, _t(table), _t(old), _t(new), f, c, co, shared_blocks=shared)
    np.testing.assert_array_equal(f.cpu().numpy(), want)
    assert co.item() == count and pool.error() == kvq.KVQ_OK
    pool.close()


@pytest.mark.parametrize("S", [6, 900])
@pytest.mark.parametrize("trouble", ["ids", "full", "negative", "row", "count"])
def test_release_of_bad_rows(S, trouble):
    rng = np.random.default_rng(S)
    bs, width = 16, 40
    old = rng.integers(0, bs * width + 1, S)
    new = rng.integers(0, 300, S)
    table = rng.permutation(S * width).reshape(S, width).astype(np.int32)
    total, cap, count = S * width, S * width + 9, 4
    if trouble == "ids":
        table[rng.random(table.shape) < 0.2] = -1
        table[rng.random(table.shape) < 0.1] = total
    elif trouble == "full":
        cap = 50
    elif trouble == "negative":
        old[0], new[1], new[2] = -5, -1, -2 ** 31
    elif trouble == "row":
        old[1] = 2 ** 31 - 1
    else:
        count = -4
    free = np.full(cap, -1, np.int32)
    want, wc, err = blocks_ref.release(table, old, new, free, count, bs, total)
    assert err
    pool = _pool(total, bs)
    f, c = _t(free), _t([count])
    kvq.kvq_release_blocks(pool.handle, _t(table), _t(old), _t(new), f, c, c)
    np.testing.assert_array_equal(f.cpu().numpy(), want)
    assert c.item() == wc and pool.error() == kvq.KVQ_ERR_OUT_OF_RANGE
    pool.close()


def test_a_captured_step_replays():
    """Release and extension captured once, in place, replayed over steps in which requests
    end and begin: every step's results are those of the walk."""
    rng = np.random.default_rng(2)
    S, bs, width, nb, rows = 12, 16, 8, 80, 40
    pool = _pool(nb, bs)
    lens, table = np.zeros(S, np.int32), np.full((S, width), -1, np.int32)
    free, count = np.full(nb, -1, np.int32), nb
    free[:] = rng.permutation(nb)
    dt, dl, dk, dn = _t(table), _t(lens), _t(lens), _t(lens)
    df, dc = _t(free), _t([count])
    q, s, p = torch.empty(S + 1, dtype=I32, device=DEV), torch.empty(rows, dtype=I64, device=DEV), torch.empty(rows, dtype=I64, device=DEV)

    def step():
        kvq.kvq_release_blocks(pool.handle, dt, dl, dk, df, dc, dc)
        dl.copy_(dk)
        kvq.kvq_extend_tables(pool.handle, dn, dt, dl, df, dc, dl, dc, q, s, p)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()  # warm-up: nothing to do yet
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for it in range(12):
        kept = np.where(rng.random(S) < 0.2, 0, lens).astype(np.int32)
        n = np.minimum(rng.integers(0, 6, S), width * bs - kept).astype(np.int32)
        dk.copy_(_t(kept))
        dn.copy_(_t(n))
        g.replay()
        free, count, err = blocks_ref.release(table, lens, kept, free, count, bs, nb)
        want, err2 = blocks_ref.extend(n, table, kept, free, count, bs, nb, rows)
        assert not err and err2 == (int(n.sum()) > rows)
        table, lens, count = want["table"], want["lens"], want["count"]
        _same({"table": dt, "lens": dl, "count": dc, "q_start": q, "slots": s, "positions": p}, want)
        np.testing.assert_array_equal(df.cpu().numpy(), free)
        held = np.concatenate([table[i, :-(-lens[i] // bs)] for i in range(S)] + [free[:count]])
        assert sorted(held) == list(range(nb))  # every block is somewhere once
    pool.close()


def test_other_streams_and_devices():
    pool = _pool(40, 16)
    table, lens, free, count = _t(np.full((2, 9), -1)), _t([0, 0]), _t(np.arange(40)), _t([40])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, s, p = pool.extend_tables(_t([20, 3]), table, lens, free, count, 30, stream=side)
    side.synchronize()
    assert q.tolist() == [0, 20, 23] and lens.tolist() == [20, 3] and count.item() == 37
    assert s[:3].tolist() == [624, 625, 626] and s[20].item() == 37 * 16 and s[23:].tolist() == [-1] * 7
    pool.release_blocks(table, lens, _t([0, 3]), free, count)
    assert count.item() == 39 and free[37:39].tolist() == [39, 38]
    with pytest.raises(ValueError, match="CUDA device"):
        pool.release_blocks(table, lens.cpu(), _t([0, 3]), free, count)
    with pytest.raises(ValueError, match="must be torch.int32"):
        pool.release_blocks(table, lens.long(), _t([0, 3]), free, count)
    pool.close()


@pytest.mark.parametrize("S,new,offset", [(3, 20, 1), (40, 100, 0), (40, 100, 1), (40, 101, 2), (600, 9, 3)])
def test_rows_at_any_address(S, new, offset):
    """Slots and positions that begin inside a larger tensor, 8 bytes off a 16-byte boundary or
    on one, calls by one CTA and by a cluster; what lies around them stays."""
    rng = np.random.default_rng(S + offset)
    lens, n, table, free, count, total = _case(rng, S, 16, 200, new, 3)
    rows = int(n.sum()) + 5
    want, err = blocks_ref.extend(n, table, lens, free, count, 16, total, rows)
    assert not err
    pool = _pool(total, 16)
    s, p = (torch.full((rows + offset + 1,), 77, dtype=I64, device=DEV) for _ in range(2))
    t, L, c, q = _t(table), _t(lens), _t([count]), torch.empty(S + 1, dtype=I32, device=DEV)
    kvq.kvq_extend_tables(pool.handle, _t(n), t, L, _t(free), c, L, c, q, s[offset:-1], p[offset:-1])
    _same({"table": t, "lens": L, "count": c, "q_start": q, "slots": s[offset:-1], "positions": p[offset:-1]}, want)
    for x in (s, p):
        assert (x[:offset] == 77).all() and x[-1] == 77
    assert pool.error() == kvq.KVQ_OK
    pool.close()


def test_sequences_without_tokens_between_distant_ones():
    """Thousands of sequences that get nothing between the few that do, and that gave nothing back."""
    S, bs = 16384, 16
    n, lens = np.zeros(S, np.int32), np.full(S, 16, np.int32)
    n[[0, 8000, S - 1]] = 1500, 40, 1500
    total = S + 200
    table = np.full((S, 100), -1, np.int32)
    table[:, 0] = np.arange(S)
    free = np.arange(S, total).astype(np.int32)
    pool = _pool(total, bs)
    want, err = blocks_ref.extend(n, table, lens, free, 200, bs, total, 3050)
    assert not err
    got = _extend(pool, n, table, lens, free, 200, 3050)
    _same(got, want)
    kept = want["lens"].copy()
    kept[[0, S - 1]] = 0
    back, count, err = blocks_ref.release(want["table"], want["lens"], kept, np.full(total, -1, np.int32), 0, bs, total)
    f, c = _t(np.full(total, -1)), _t([0])
    kvq.kvq_release_blocks(pool.handle, got["table"], got["lens"], _t(kept), f, c, c)
    np.testing.assert_array_equal(f.cpu().numpy(), back)
    assert c.item() == count and not err and pool.error() == kvq.KVQ_OK
    pool.close()


def test_many_bad_rows_in_a_cluster():
    """Ids outside the pool all over a table that a cluster frees, more of them than a turn of its
    threads: none given back, the others in order; and a list that is too short."""
    rng = np.random.default_rng(8)
    S, bs, width = 40, 16, 700
    old = rng.integers(0, width * bs + 1, S)
    old[7] = width * bs + 9  # beyond the row
    table = rng.integers(-3, 20000, (S, width)).astype(np.int32)
    total = 18000
    for capacity in (40000, 9000):
        free = np.full(capacity, -1, np.int32)
        want, count, err = blocks_ref.release(table, old, np.zeros(S, int), free, 4, bs, total)
        assert err
        pool = _pool(total, bs)
        f, c = _t(free), _t([4])
        kvq.kvq_release_blocks(pool.handle, _t(table), _t(old), _t(np.zeros(S)), f, c, c)
        np.testing.assert_array_equal(f.cpu().numpy(), want)
        assert c.item() == count and pool.error() == kvq.KVQ_ERR_OUT_OF_RANGE
        pool.close()


def test_evicted_blocks_come_back():
    """An eviction's tables and lengths are what a release takes: the evicted blocks come back, the
    kept ones stay, and every block is somewhere once."""
    rng = np.random.default_rng(5)
    S, bs, nb, budget = 4, 16, 64, 5
    lens = np.array([200, 33, 0, 81], np.int32)
    per = -(-lens // bs)
    ids = rng.permutation(nb).astype(np.int32)
    table = np.full((S, 14), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(per)])
    for s in range(S):
        table[s, :per[s]] = ids[at[s]:at[s + 1]]
    free = np.full(nb, -1, np.int32)
    free[:nb - at[-1]] = ids[at[-1]:]
    pool = _pool(nb, bs)
    scores = torch.rand((S, 1, 14 * bs), device=DEV)
    t2, l2, kept, _ = pool.evict_blocks(scores, _t(table), _t(lens), 200, budget, sink_blocks=1)
    f, c = _t(free), _t([nb - at[-1]])
    pool.release_blocks(t2, _t(lens), l2, f, c)
    new, t2 = l2.cpu().numpy(), t2.cpu().numpy()
    held = -(-new // bs)
    assert (held == np.minimum(per, budget)).all() and c.item() == nb - held.sum()
    here = np.concatenate([t2[s, :held[s]] for s in range(S)] + [f.cpu().numpy()[:c.item()]])
    assert sorted(here) == list(range(nb))
    for s in range(S):
        assert set(t2[s, :held[s]]) <= set(table[s, :per[s]])
    assert pool.error() == kvq.KVQ_OK
    pool.close()
