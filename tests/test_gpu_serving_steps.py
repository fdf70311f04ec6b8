"""Serving steps as a program makes them: blocks come back and are given out on the GPU, the
slot map that comes out feeds two layers' 4-bit pools (rotated keys and ordinary attention
in one, differential attention in the other), prompts and single tokens in turn, by calls
and by captured graphs that share a workspace."""
import numpy as np
import pytest
import torch

import blocks_ref
import paged_quantized_kv_kvq_gb300 as kvq
from cache_ops_ref import attention, frequencies, rope, tokens
from fp4_ref import quantize, values

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
S, BS, NB, WIDTH, HQ, HKV, D = 5, 16, 60, 14, 8, 2, 128
MOST = WIDTH * BS
I32, I64 = torch.int32, torch.int64


def _t(x, dtype=None):
    x = torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
    return x if dtype is None else x.to(dtype)


class Loop:
    """The device state of the steps, and the same state as a plain walk keeps it."""

    def __init__(self, rows, seed):
        self.rng, self.rows = np.random.default_rng(seed), rows
        self.pools = [kvq.KVPool(NB, BS, HKV, D, kvq.KVQ_FP4_E2M1, device=DEV, fill_byte=0xFF) for _ in range(2)]
        self.rope = kvq.kvq_rope_init(D)
        self.lens, self.table = np.zeros(S, np.int32), np.full((S, WIDTH), -1, np.int32)
        self.free, self.count = self.rng.permutation(NB).astype(np.int32), NB
        self.dt, self.dl, self.df, self.dc = _t(self.table), _t(self.lens), _t(self.free), _t(np.array([NB], np.int32))
        self.kept, self.new = _t(self.lens), _t(self.lens)
        self.q_start = torch.empty(S + 1, dtype=I32, device=DEV)
        self.slots, self.pos = (torch.empty(rows, dtype=I64, device=DEV) for _ in range(2))
        self.q, self.k, self.v = (torch.empty((rows, h, D), dtype=torch.float16, device=DEV) for h in (HQ, HKV, HKV))
        self.lam, self.w = _t(self.rng.uniform(0, 0.8, HQ).astype(np.float32)), _t(self.rng.uniform(0.5, 1.5, D).astype(np.float32))
        self.rq = torch.zeros_like(self.q)
        need = [kvq.kvq_prefill_workspace_bytes(self.pools[0].handle, S, MOST), kvq.kvq_decode_workspace_bytes(self.pools[0].handle, S, HQ, MOST),
                kvq.kvq_diff_prefill_workspace_bytes(self.pools[1].handle, S, rows, HQ, MOST),
                kvq.kvq_diff_decode_workspace_bytes(self.pools[1].handle, S, HQ, MOST)]
        self.ws = torch.full((max(need),), 0xFF, dtype=torch.uint8, device=DEV)
        self.out = torch.empty((rows, HQ, D), device=DEV)
        self.diff = torch.empty((rows, HQ, D), dtype=torch.float16, device=DEV)

    def close(self):
        for p in self.pools:
            assert p.error() == kvq.KVQ_OK
            p.close()

    def plan(self, kept, n):
        """The next step's inputs on the device, and the walk's answer."""
        self.kept.copy_(_t(kept))
        self.new.copy_(_t(n))
        for x in (self.q, self.k, self.v):
            x.copy_(_t(self.rng.standard_normal(x.shape).astype(np.float16)))
        self.out.fill_(7)
        self.diff.fill_(7)
        self.free, self.count, err = blocks_ref.release(self.table, self.lens, kept, self.free, self.count, BS, NB)
        assert not err
        self.want, err = blocks_ref.extend(n, self.table, kept, self.free, self.count, BS, NB, self.rows)
        assert not err
        self.table, self.lens, self.count = self.want["table"], self.want["lens"], self.want["count"]

    def step(self, most_new):
        a, b = (p.handle for p in self.pools)
        kvq.kvq_release_blocks(a, self.dt, self.dl, self.kept, self.df, self.dc, self.dc)
        self.dl.copy_(self.kept)
        kvq.kvq_extend_tables(a, self.new, self.dt, self.dl, self.df, self.dc, self.dl, self.dc, self.q_start, self.slots, self.pos)
        kvq.kvq_rope_append(a, self.rope, self.q, self.k, self.v, self.pos, self.slots, self.rq)
        kvq.kvq_append(b, self.k, self.v, self.slots)
        if most_new == 1:  # every sequence has one row
            kvq.kvq_paged_decode(a, self.rq[:S], self.dt, self.dl, MOST, D ** -0.5, self.out[:S], self.ws)
            kvq.kvq_diff_decode(b, self.q[:S], self.dt, self.dl, MOST, (D // 2) ** -0.5, self.lam, self.diff[:S], self.ws, self.w, 1e-5, 0.5)
        else:
            kvq.kvq_prefill_ex(a, self.rq, self.q_start, most_new, self.dt, self.dl, MOST, D ** -0.5, self.out, self.ws)
            kvq.kvq_diff_prefill(b, self.q, self.q_start, most_new, self.dt, self.dl, MOST, (D // 2) ** -0.5, self.lam, self.diff, self.ws,
                                 self.w, 1e-5, 0.5)

    def check(self):
        torch.cuda.synchronize()
        for name, got in (("table", self.dt), ("lens", self.dl), ("count", self.dc), ("q_start", self.q_start), ("slots", self.slots),
                          ("positions", self.pos)):
            np.testing.assert_array_equal(got.cpu().numpy().reshape(np.shape(self.want[name])), self.want[name], err_msg=name)
        np.testing.assert_array_equal(self.df.cpu().numpy(), self.free)
        held = [self.table[s, :-(-self.lens[s] // BS)] for s in range(S)]
        assert sorted(np.concatenate(held + [self.free[:self.count]])) == list(range(NB))  # every block is somewhere once
        start = self.want["q_start"]
        T = int(start[-1])
        assert (self.out[T:] == 7).all() and (self.diff[T:] == 7).all()
        if T == 0:
            return
        at, pos = self.want["slots"][:T], self.want["positions"][:T]
        k, v = self.k[:T].cpu().numpy(), self.v[:T].cpu().numpy()
        # layer 0: the rotated keys, within half of the codes' largest step, 2, at a scale that is
        # absmax / 6 within 1/16: 0.18 of absmax (what that saturates is off by 1/16 at most)
        y = rope(k, pos, frequencies(D))
        got = [x.double().cpu().numpy() for x in self.pools[0].read_values(_t(at))]
        group = np.abs(y).reshape(T, HKV, -1, 16).max(-1).repeat(16, -1)
        assert (np.abs(got[0] - y) <= 0.18 * group).all()
        np.testing.assert_array_equal(got[1], values(*quantize(v)))
        # layer 1: the rows as they came
        got = [x.double().cpu().numpy() for x in self.pools[1].read_values(_t(at))]
        np.testing.assert_array_equal(got[0], values(*quantize(k)))
        np.testing.assert_array_equal(got[1], values(*quantize(v)))
        # attention of every row over what the pools say they hold
        seq = np.repeat(np.arange(S), np.diff(start))
        rows = (pos + 1).astype(np.int32)
        held = [torch.stack(p.read_values(torch.arange(NB * BS, device=DEV)), 1).double().cpu().numpy() for p in self.pools]
        rq = self.rq[:T].double().cpu().numpy()
        q = self.q[:T].cpu().numpy()
        want = attention(lambda r: held[0][tokens(self.table[seq], rows, r, BS)], rq, rows, D ** -0.5)[0]
        np.testing.assert_allclose(rq, rope(q, pos, frequencies(D)), rtol=2.0 ** -10, atol=2.0 ** -8)
        out = self.out[:T].cpu().numpy()
        # exact dequantized values, fp32 sums and weights within 2^-22: 1e-5 as a whole
        assert np.linalg.norm(out - want) <= 1e-5 * np.linalg.norm(want)
        maps = []
        for a, b in ((0, D // 2), (D // 2, D)):
            def half(r):
                x = held[1][tokens(self.table[seq], rows, r, BS)].copy()
                x[:, 0, :, :a] = 0
                x[:, 0, :, b:] = 0
                return x

            maps.append(attention(half, q, rows, (D // 2) ** -0.5)[0])
        lam, w = self.lam.double().cpu().numpy()[None, :, None], self.w.double().cpu().numpy()
        d = maps[0] - lam * maps[1]
        rms = np.sqrt((d * d).mean(-1, keepdims=True) + 1e-5)
        want = d / rms * w * 0.5
        # half a step of fp16; the error e of the difference (a prompt's fp16 weights, each within 2^-11 of
        # itself, in the sum of values and in what divides it), and what the norm makes of it: e / rms
        # from the value, |d| / rms times as much from the root mean square
        size = np.abs(maps[0]).max(-1, keepdims=True) + np.abs(lam) * np.abs(maps[1]).max(-1, keepdims=True)
        peak = max(np.abs(held[1][tokens(self.table, self.lens, s, BS), 1]).max(initial=0) for s in range(S))
        e = 2.0 ** -11 * (size + (1 + np.abs(lam)) * peak)
        bound = np.abs(want) * 2.0 ** -11 + e / rms * (1 + np.abs(d) / rms) * w.max() * 0.5 + 2.0 ** -25
        assert (np.abs(self.diff[:T].double().cpu().numpy() - want) <= bound).all()


def _requests(loop, it):
    """Prompts on every third step, single tokens between them."""
    rng = loop.rng
    if it % 3 == 0:
        kept = np.where((rng.random(S) < 0.4) | (loop.lens > MOST - 80), 0, loop.lens).astype(np.int32)
        n = np.where(kept == 0, rng.integers(1, 61, S), rng.integers(0, 4, S)).astype(np.int32)
        return kept, n, 60
    return loop.lens.copy(), np.ones(S, np.int32), 1


def test_steps():
    loop = Loop(5 * 60 + 3, seed=1)
    for it in range(7):
        kept, n, most = _requests(loop, it)
        loop.plan(kept, n)
        loop.step(most)
        loop.check()
    loop.close()


def test_captured_steps_share_a_workspace():
    """A graph of a prompt's step and one of single tokens over the same buffers, replayed in turn."""
    loop = Loop(5 * 60, seed=2)
    side = torch.cuda.Stream()
    for most in (60, 1):  # warm-up: nothing to do yet
        loop.plan(np.zeros(S, np.int32), np.zeros(S, np.int32))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            loop.step(most)
        torch.cuda.synchronize()
    graphs = {}
    for most in (60, 1):
        graphs[most] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[most], stream=side):
            loop.step(most)
    for it in range(9):
        kept, n, most = _requests(loop, it)
        loop.plan(kept, n)
        torch.cuda.synchronize()
        graphs[most].replay()
        loop.check()
    loop.close()


def test_steps_of_two_programs_at_once():
    """Two programs with pools and workspaces of their own, on two streams at the same time."""
    loops, sides = [Loop(5 * 60, seed=3), Loop(5 * 60, seed=4)], [torch.cuda.Stream() for _ in range(2)]
    for it in range(4):
        work = [_requests(loop, it) for loop in loops]
        for loop, (kept, n, _) in zip(loops, work):
            loop.plan(kept, n)
        torch.cuda.synchronize()
        for side in sides:
            with torch.cuda.stream(side):
                torch.cuda._sleep(2_000_000)
        for loop, side, (_, _, most) in zip(loops, sides, work):
            with torch.cuda.stream(side):
                loop.step(most)
        for loop in loops:
            loop.check()
    for loop in loops:
        loop.close()
