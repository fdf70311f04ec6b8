"""Timing cases of block bookkeeping, the 4-bit cache and differential attention.

Four operators, each with its plain form in elementary torch operations
(`own` false) and as calls of this package (`own` true):

  blocks   a serving step's block tables, slot map and positions from the requests' lengths
  append4  keys and values quantized into a cache of 4-bit floats with a scale per 16 channels
  attend4  attention over that cache: single tokens, and prompts
  diff     differential attention over a paged cache: single tokens, and prompts
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-5
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # of the 4-bit float's codes 0 .. 7; 8 .. 15 are their negatives

# cache format -> the package's constant and bits per element
FORMATS = {"fp4": ("KVQ_FP4_E2M1", 4), "int8_block": ("KVQ_INT8_PER_BLOCK", 8), "e4m3_block": ("KVQ_FP8_E4M3_PER_BLOCK", 8)}


def listed():
    return [
        # a decode step of 64 sequences: a few have ended, as many begin with short prompts, the others take a token each (latency)
        {"name": "blocks_step", "op": "blocks", "S": 64, "L": 2048, "ended": 4, "begun": 4, "n": 100, "bs": 16},
        # a step that takes in prompts: 512 rows, an eighth of them new, up to 1024 tokens each
        {"name": "blocks_prompts", "op": "blocks", "S": 512, "L": 4000, "ended": 64, "begun": 64, "n": 1024, "bs": 16},
        # a decode step's new tokens of 64 sequences, all over their blocks
        {"name": "append4_step", "op": "append4", "S": 64, "n": 1, "at": 3, "hkv": 8, "d": 128, "bs": 16},
        # prompts of 8 x 2048 tokens
        {"name": "append4_prompt", "op": "append4", "S": 8, "n": 2048, "at": 0, "hkv": 8, "d": 128, "bs": 16},
        # four short requests (latency)
        {"name": "attend4_tiny", "op": "attend4", "S": 4, "L": 100, "n": 1, "ragged": True, "hq": 4, "hkv": 1, "d": 64, "bs": 16},
        # the serving batch: 64 sequences of 2048 tokens
        {"name": "attend4_batch", "op": "attend4", "S": 64, "L": 2048, "n": 1, "ragged": False, "hq": 32, "hkv": 8, "d": 128, "bs": 16},
        # long contexts in larger blocks, lengths that differ
        {"name": "attend4_long", "op": "attend4", "S": 8, "L": 32768, "n": 1, "ragged": True, "hq": 32, "hkv": 8, "d": 128, "bs": 32},
        # whole prompts of 8 x 2048 tokens
        {"name": "attend4_prompt", "op": "attend4", "S": 8, "L": 2048, "n": 2048, "ragged": False, "hq": 32, "hkv": 8, "d": 128, "bs": 16},
        # a few short requests (latency): 8 differential heads over 2 kv heads, each kv head's keys in two halves
        {"name": "diff_tiny", "op": "diff", "S": 5, "L": 77, "n": 1, "ragged": True, "hq": 8, "hkv": 2, "d": 128, "norm": True,
         "fmt": "int8_block", "bs": 16},
        # the serving batch over 8-bit blocks
        {"name": "diff_batch", "op": "diff", "S": 64, "L": 2048, "n": 1, "ragged": False, "hq": 16, "hkv": 8, "d": 128, "norm": True,
         "fmt": "int8_block", "bs": 16},
        # long contexts over the 4-bit cache
        {"name": "diff_long", "op": "diff", "S": 8, "L": 32768, "n": 1, "ragged": True, "hq": 16, "hkv": 8, "d": 128, "norm": True,
         "fmt": "fp4", "bs": 32},
        # whole prompts over the 4-bit cache
        {"name": "diff_prompt", "op": "diff", "S": 8, "L": 2048, "n": 2048, "ragged": False, "hq": 16, "hkv": 4, "d": 128, "norm": True,
         "fmt": "fp4", "bs": 16},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["blocks", "append4", "append4", "attend4", "attend4", "attend4", "diff", "diff", "diff"])
    bs = rng.choice([16, 32, 64])
    if op == "blocks":
        S = _log(rng, 1, 512)
        ended = rng.randint(0, S // 4)
        begun = rng.randint(0, S // 4)
        return {"op": op, "S": S, "L": _log(rng, 1, 4000), "ended": ended, "begun": begun,
                "n": _log(rng, 1, min(4096, 65536 // max(1, begun))), "bs": rng.choice([8, bs])}
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 8, 32])
    if op == "append4":
        most = min(16384, 16384 * 8 * 128 // (hkv * d))
        if rng.random() < 0.5:
            return {"op": op, "S": _log(rng, 1, min(256, most)), "n": 1, "at": rng.randint(0, bs - 1), "hkv": hkv, "d": d, "bs": bs}
        S = _log(rng, 1, 16)
        return {"op": op, "S": S, "n": _log(rng, 2, max(3, most // S)), "at": rng.choice([0, 0, rng.randint(1, bs - 1)]), "hkv": hkv,
                "d": d, "bs": bs}
    hq = hkv * (rng.choice([1, 2, 3, 4, 8]) if hkv < 32 else 1)
    c = {"op": op, "S": 1, "L": 1, "n": 1, "ragged": rng.random() < 0.7, "hq": hq, "hkv": hkv, "d": d, "bs": bs}
    if rng.random() < 0.7:
        c["S"] = _log(rng, 1, 128)
        c["L"] = _log(rng, 17, min(32768, 8 * 32768 * 8 * 128 // (c["S"] * max(hkv, hq // 4) * d)))
    else:
        c["S"] = _log(rng, 1, 8)
        c["L"] = _log(rng, 17, min(2048, 16384 * 16 * 128 // (c["S"] * hq * d)))
        c["n"] = rng.choice([c["L"], rng.randint(2, c["L"])])
    if op == "diff":
        c["norm"], c["fmt"] = rng.random() < 0.7, rng.choice(["fp4", "fp4", "int8_block", "e4m3_block"])
    return c


def _spread(most, count):
    """`count` whole numbers over 1 .. most, the first of them `most`."""
    return [1 + int((most - 1) * (1.0 - (s * 0.6180339887498949) % 1.0)) for s in range(count)]


def _lens(c):
    return _spread(c["L"], c["S"]) if c["ragged"] else [c["L"]] * c["S"]


def _news(c):
    """New tokens of each sequence, the last ones of its cached tokens."""
    return [min(n, c["n"]) for n in _lens(c)]


# ------------------------------------------------------------------ work
def _cache_bytes(fmt, d, hkv, tokens, blocks):
    bits = FORMATS[fmt][1]
    return 2 * (tokens * hkv * d * bits // 8 + (tokens * hkv * d // 16 if fmt == "fp4" else blocks * hkv * 4))


def work(c):
    op = c["op"]
    if op == "blocks":
        lens, kept, n = _step_lens(c)
        bs = c["bs"]
        freed = sum(-(-a // bs) - -(-b // bs) for a, b in zip(lens, kept))
        taken = sum(-(-(a + b) // bs) - -(-a // bs) for a, b in zip(kept, n))
        tail = sum(1 for a, b in zip(kept, n) if b and a % bs)  # a partly filled block whose id is looked up
        return {"bytes": 8 * freed + 8 * taken + 4 * tail + 20 * c["S"] + 16 * sum(n), "flops": 4 * sum(n) + 4 * c["S"]}
    if op == "append4":
        kv = c["S"] * c["n"] * c["hkv"] * c["d"]
        # tokens in, codes and scales out, and the same read back as fp16
        return {"bytes": 4 * kv + 2 * _cache_bytes("fp4", c["d"], c["hkv"], c["S"] * c["n"], 0) + 4 * kv + 16 * c["S"] * c["n"],
                "flops": 6 * kv}
    lens, news = _lens(c), _news(c)
    tokens, blocks = sum(lens), sum(-(-n // c["bs"]) for n in lens)
    pairs = sum(n * (L - n) + n * (n + 1) // 2 for L, n in zip(lens, news))
    rows = sum(news) * c["hq"] * c["d"]
    if op == "attend4":
        return {"bytes": _cache_bytes("fp4", c["d"], c["hkv"], tokens, blocks) + 6 * rows + 4 * blocks,
                "flops": 4 * pairs * c["hq"] * c["d"]}
    return {"bytes": _cache_bytes(c["fmt"], c["d"], c["hkv"], tokens, blocks) + 4 * rows + 4 * blocks,
            "flops": 6 * pairs * c["hq"] * c["d"]}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _step_lens(c):
    """Cached tokens before the step, after the ended sequences' blocks are given back, and the step's new tokens."""
    S, ended, begun = c["S"], c["ended"], c["begun"]
    lens = _spread(c["L"], S)
    lens[S - begun:] = [0] * begun  # rows that wait for a request
    kept = [0] * ended + lens[ended:]
    n = [0] * ended + [1] * (S - ended - begun) + _spread(c["n"], begun)
    return lens, kept, n


def _div(a, b):
    """IEEE a / b with zeros where b is zero (a divisor that is a plain number may be multiplied by instead)."""
    return torch.where(b == 0, torch.zeros_like(a), a / torch.where(b == 0, torch.ones_like(b), b))


def _const(x, like):
    return torch.full((), x, device=DEV, dtype=like.dtype)


def _micro_scale(amax):
    """amax / 6 in 8 bits: 3 of mantissa, exponents -14 .. 15 with subnormals below, at most 10240 so that 6 of it is an fp16 value."""
    y = amax / _const(6.0, amax)
    low = y.clamp(min=2.0 ** -14)
    step = low / torch.frexp(low)[0] / _const(16.0, y)  # powers of two
    return (torch.round(y / step) * step).clamp(max=10240.0)


def _micro_codes(x):
    """(codes 0 .. 15, scales as numbers) of x [..., d]: a scale per 16 channels, codes to nearest with ties to the even one."""
    x = x.unflatten(-1, (-1, 16))
    s = _micro_scale(x.abs().amax(-1, keepdim=True))
    q = _div(x, s.expand_as(x))
    a = q.abs()
    code = sum((a > b).to(torch.uint8) for b in (0.25, 1.25, 2.5, 5.0)) + sum((a >= b).to(torch.uint8) for b in (0.75, 1.75, 3.5))
    code = code + 8 * (torch.signbit(q) & (code > 0)).to(torch.uint8)
    return code.flatten(-2), s.squeeze(-1)


def _micro_values(code, s, dtype):
    """code * scale in `dtype`."""
    m = torch.tensor([*MAGNITUDES, *(-v for v in MAGNITUDES)], device=DEV, dtype=dtype)
    return (m[code.int()].unflatten(-1, (-1, 16)) * s.to(dtype).unsqueeze(-1)).flatten(-2)


def _block_codes(x, fmt):
    """(codes, scales) of blocks x [N, bs, H, D] with one scale for each block and head."""
    top = 448.0 if fmt == "e4m3_block" else 127.0
    s = x.abs().amax((1, 3), keepdim=True) / _const(top, x)
    y = _div(x, s.expand_as(x))
    if fmt == "e4m3_block":
        return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), s
    return y.round().clamp(-127.0, 127.0).to(torch.int8), s


def _cache(c, seed):
    """A filled cache: fp16 tokens K, V [N, bs, H, D], their codes and scales, the block table, the lengths and the queries."""
    g = _gen(seed)
    S, hkv, d, bs, fmt = c["S"], c["hkv"], c["d"], c["bs"], c.get("fmt", "fp4")
    lens, news = _lens(c), _news(c)
    nb = -(-c["L"] // bs)
    N = S * nb
    gain = 1.0 + 9.0 * (torch.rand(hkv * d, generator=g, device=DEV) < 0.01)
    perm = torch.randperm(N, generator=g, device=DEV).to(torch.int32)
    at = torch.arange(nb * bs, device=DEV).view(1, nb, bs)
    s = {"case": c, "table": perm.view(S, nb), "lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "blocks": N,
         "q": _randn(g, sum(news), c["hq"], d).half(), "q_start": torch.tensor(np.cumsum([0] + news), dtype=torch.int32, device=DEV)}
    filled = torch.zeros((N, bs), dtype=torch.bool, device=DEV)
    filled[perm.long()] = (at < s["lens"].view(S, 1, 1)).view(N, bs)
    for x in ("k", "v"):
        t = (_randn(g, N, bs, hkv * d) * gain).half().view(N, bs, hkv, d) * filled.view(N, bs, 1, 1)
        s[x] = t
        s[x + "c"], s[x + "s"] = _micro_codes(t.float()) if fmt == "fp4" else _block_codes(t.float(), fmt)
    s["filled"] = filled
    s["scale"] = (d // 2 if c["op"] == "diff" else d) ** -0.5
    if c["op"] == "diff":
        s["lambda"] = 0.2 + 0.6 * torch.rand(c["hq"], generator=g, device=DEV)
        s["weight"] = 1.0 + 0.1 * _randn(g, d) if c["norm"] else None
        s["out_scale"] = 0.2 if c["norm"] else 1.0
    return s


def _values(s, x, i, dtype):
    """The cache of x ("k" or "v") along sequence i (all of them: a slice), in `dtype`: [S, tokens, H, D]."""
    at = s["table"][i].long()
    code, sc = s[x + "c"], s[x + "s"]
    if code.dtype == torch.uint8:
        return _micro_values(code[at], sc[at], dtype).flatten(1, 2)
    y = code.view(torch.uint8)[at].view(code.dtype) if code.dtype == torch.float8_e4m3fn else code[at]
    return (y.to(dtype) * sc[at].to(dtype)).flatten(1, 2)


def _fill_pool(s, c):
    """The package's pool with the same tokens."""
    import paged_quantized_kv_kvq_gb300 as kvq

    pool = kvq.KVPool(s["blocks"], c["bs"], c["hkv"], c["d"], getattr(kvq, FORMATS[c.get("fmt", "fp4")][0]), device=DEV)
    slots = torch.arange(s["blocks"] * c["bs"], device=DEV)
    pool.append(s["k"].flatten(0, 1), s["v"].flatten(0, 1), torch.where(s["filled"].view(-1), slots, -1))
    return pool


def _prepare_blocks(c, seed):
    lens, kept, n = _step_lens(c)
    bs, S = c["bs"], c["S"]
    r = np.random.RandomState(seed % (1 << 31))
    held = [-(-x // bs) for x in lens]
    width = max(max(-(-(a + b) // bs) for a, b in zip(kept, n)), max(held), 1) + 2
    spare = sum(-(-(a + b) // bs) for a, b in zip(kept, n)) + 5
    N = sum(held) + spare
    ids = r.permutation(N).astype(np.int32)
    table = np.full((S, width), -1, np.int32)
    at = 0
    for s, h in enumerate(held):
        table[s, :h] = ids[at:at + h]
        at += h
    free = np.full(N, -1, np.int32)
    free[:spare] = ids[at:]
    put = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return {"case": c, "table": put(table), "lens": put(lens), "kept": put(kept), "n": put(n), "free": put(free), "count": put([spare]),
            "blocks": N, "rows": sum(n)}


def prepare(c, seed):
    op = c["op"]
    if op == "blocks":
        s = _prepare_blocks(c, seed)
        if own:
            import paged_quantized_kv_kvq_gb300 as kvq

            s["kvq"] = kvq
            s["pool"] = kvq.KVPool(s["blocks"], c["bs"], 1, 64, kvq.KVQ_FP8_E5M2, device=DEV)
            s["freed"], s["left"] = torch.empty_like(s["count"]), torch.empty_like(s["count"])
            s["lens_out"] = torch.empty_like(s["lens"])
            s["q_start"] = torch.empty(c["S"] + 1, dtype=torch.int32, device=DEV)
            s["slots"] = torch.empty(s["rows"], dtype=torch.int64, device=DEV)
            s["positions"] = torch.empty_like(s["slots"])
        return s
    if op == "append4":
        g = _gen(seed)
        T, hkv, d, bs = c["S"] * c["n"], c["hkv"], c["d"], c["bs"]
        gain = 1.0 + 9.0 * (torch.rand(hkv * d, generator=g, device=DEV) < 0.01)
        s = {"case": c, "k": (_randn(g, T, hkv * d) * gain).half().view(T, hkv, d), "v": (_randn(g, T, hkv * d) * gain).half().view(T, hkv, d)}
        first = (7 * np.arange(c["S"]) + c["at"]) % bs if c["n"] == 1 else np.full(c["S"], c["at"])
        per = (c["at"] + c["n"] + bs - 1) // bs if c["n"] > 1 else 1
        blocks = np.random.RandomState(seed % (1 << 31)).permutation(c["S"] * per + 3)[:c["S"] * per].reshape(c["S"], per)
        t = first[:, None] + np.arange(c["n"])
        s["slots"] = torch.from_numpy((np.take_along_axis(blocks, t // bs, 1) * bs + t % bs).reshape(-1)).to(DEV)
        if own:
            import paged_quantized_kv_kvq_gb300 as kvq

            s["kvq"] = kvq
            s["pool"] = kvq.KVPool(c["S"] * per + 3, bs, hkv, d, kvq.KVQ_FP4_E2M1, device=DEV)
            s["k_values"], s["v_values"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        return s
    s = _cache(c, seed)
    if own:
        import paged_quantized_kv_kvq_gb300 as kvq

        s["kvq"], s["pool"] = kvq, _fill_pool(s, c)
        h, S, T = s["pool"].handle, c["S"], s["q"].shape[0]
        if op == "attend4":
            ws = kvq.kvq_decode_workspace_bytes(h, S, c["hq"], c["L"]) if c["n"] == 1 else kvq.kvq_prefill_workspace_bytes(h, S, c["L"])
        elif c["n"] == 1:
            ws = kvq.kvq_diff_decode_workspace_bytes(h, S, c["hq"], c["L"])
        else:
            ws = kvq.kvq_diff_prefill_workspace_bytes(h, S, T, c["hq"], c["L"])
        s["ws"] = torch.empty(max(ws, 1), dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty((T, c["hq"], c["d"]), dtype=torch.float32 if op == "attend4" else torch.float16, device=DEV)
    del s["k"], s["v"], s["filled"]  # the fp16 tokens themselves are no part of the cache
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    c, kvq = s["case"], s["kvq"]
    h = s["pool"].handle
    if c["op"] == "blocks":
        kvq.kvq_release_blocks(h, s["table"], s["lens"], s["kept"], s["free"], s["count"], s["freed"])
        kvq.kvq_extend_tables(h, s["n"], s["table"], s["kept"], s["free"], s["freed"], s["lens_out"], s["left"], s["q_start"], s["slots"],
                              s["positions"])
        return {"table": s["table"], "lens": s["lens_out"], "free": s["free"], "freed": s["freed"], "left": s["left"], "q_start": s["q_start"],
                "slots": s["slots"], "positions": s["positions"]}
    if c["op"] == "append4":
        kvq.kvq_append(h, s["k"], s["v"], s["slots"])
        kvq.kvq_read_values(h, s["slots"], s["k_values"], s["v_values"])
        return {"k": s["k_values"], "v": s["v_values"]}
    if c["op"] == "attend4":
        if c["n"] == 1:
            kvq.kvq_paged_decode(h, s["q"], s["table"], s["lens"], c["L"], s["scale"], s["out"], s["ws"])
        else:
            kvq.kvq_prefill_ex(h, s["q"], s["q_start"], c["n"], s["table"], s["lens"], c["L"], s["scale"], s["out"], s["ws"])
        return s["out"]
    if c["n"] == 1:
        kvq.kvq_diff_decode(h, s["q"], s["table"], s["lens"], c["L"], s["scale"], s["lambda"], s["out"], s["ws"], s["weight"], EPS, s["out_scale"])
    else:
        kvq.kvq_diff_prefill(h, s["q"], s["q_start"], c["n"], s["table"], s["lens"], c["L"], s["scale"], s["lambda"], s["out"], s["ws"],
                             s["weight"], EPS, s["out_scale"])
    return s["out"]


def _plain(s):
    c = s["case"]
    if c["op"] == "blocks":
        return _plain_blocks(s)
    if c["op"] == "append4":
        return {x: _micro_values(*_micro_codes(s[x].float()), torch.float32).half() for x in ("k", "v")}
    hkv, S, n, L = c["hkv"], c["S"], c["n"], c["L"]
    k, v = (_values(s, x, slice(None), torch.float32)[:, :L].transpose(1, 2) for x in ("k", "v"))  # [S, H, tokens, D]
    lens = s["lens"].long()
    # rows of a sequence beside each other, those that a shorter one lacks repeated and dropped at the end
    news = (s["q_start"][1:] - s["q_start"][:-1]).long()
    i = torch.arange(n, device=DEV)
    there = i < news.view(S, 1)
    row = s["q_start"][:-1].long().view(S, 1) + torch.minimum(i, news.view(S, 1) - 1)
    q = s["q"][row].float().transpose(1, 2).unflatten(1, (hkv, -1))  # [S, H, group, n, D]
    past = torch.arange(L, device=DEV) > (lens - news).view(S, 1, 1) + i.view(1, n, 1)
    past = (past | (torch.arange(L, device=DEV) >= lens.view(S, 1, 1))).view(S, 1, 1, n, L)

    def attend(q, k):
        z = (torch.matmul(q.flatten(2, 3), k.transpose(2, 3)) * s["scale"]).view(S, hkv, -1, n, L)
        z.masked_fill_(past, -math.inf)
        z = torch.exp(z - z.amax(-1, keepdim=True))
        z /= z.sum(-1, keepdim=True)
        return torch.matmul(z.flatten(2, 3), v).view(S, hkv, -1, n, c["d"])

    if c["op"] == "attend4":
        return attend(q, k).flatten(1, 2).transpose(1, 2)[there]
    half = c["d"] // 2
    y = attend(q[..., :half], k[..., :half])
    y = (y - s["lambda"].view(1, hkv, -1, 1, 1) * attend(q[..., half:], k[..., half:])).flatten(1, 2).transpose(1, 2)[there]
    if s["weight"] is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    return (y * s["out_scale"]).half()


def _plain_blocks(s):
    c = s["case"]
    bs, S, rows = c["bs"], c["S"], s["rows"]
    lens, kept, n, table, free = s["lens"].long(), s["kept"].long(), s["n"].long(), s["table"].clone(), s["free"].clone()
    up = lambda x: (x + bs - 1) // bs  # noqa: E731
    j = torch.arange(table.shape[1], device=DEV)
    # the blocks given back, in the order of their sequences, behind the free ones
    gone = table[(j >= up(kept).view(S, 1)) & (j < up(lens).view(S, 1))]
    count = s["count"] + gone.numel()
    free[s["count"].long() + torch.arange(gone.numel(), device=DEV)] = gone
    # blocks taken from the end of the list
    need = up(kept + n) - up(kept)
    before = torch.cumsum(need, 0) - need
    k = before.view(S, 1) + j - up(kept).view(S, 1)
    new = (j >= up(kept).view(S, 1)) & (j < up(kept + n).view(S, 1))
    table = torch.where(new, free[(count.long() - 1 - k).clamp(min=0)], table)
    q_start = torch.cat((torch.zeros_like(n[:1]), torch.cumsum(n, 0)))
    r = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(q_start[1:].contiguous(), r, right=True)
    pos = kept[seq] + r - q_start[seq]
    return {"table": table, "lens": (kept + n).int(), "free": free, "freed": count, "left": count - need.sum().int(), "q_start": q_start.int(),
            "slots": table[seq, pos // bs].long() * bs + pos % bs, "positions": pos}


# ------------------------------------------------------------------ the definitions in 64 bits
def _nearest4(x):
    """x [..., d] in groups of 16 as the nearest 4-bit floats at the groups' scales."""
    y = x.reshape(*x.shape[:-1], -1, 16)
    want = (y.abs().amax(-1, keepdim=True) / 6.0).float().double()
    e = torch.floor(torch.log2(want.clamp(min=2.0 ** -14))).clamp(max=15).long()
    step = torch.tensor([2.0 ** (i - 3) for i in range(-14, 16)], dtype=torch.float64, device=DEV)[e + 14]
    s = torch.minimum(torch.round(want / step) * step, torch.full_like(want, 10240.0))
    q = y / torch.where(s > 0, s, torch.ones_like(s))
    a = q.abs()
    a = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2)).clamp(max=6.0)
    return torch.where(s > 0, a * torch.sign(q) * s, torch.zeros_like(y)).reshape(x.shape)


def exact(c, seed):
    if c["op"] == "blocks":  # whole numbers
        return None
    if c["op"] == "append4":
        s = prepare(c, seed)
        return {x: _nearest4(s[x].double()) for x in ("k", "v")}
    s = _cache(c, seed)
    fmt, d = c.get("fmt", "fp4"), c["d"]
    outs, at = [], 0
    for i, (L, n) in enumerate(zip(_lens(c), _news(c))):  # one sequence after the other: 64 bits of a long one fill some memory
        where = s["table"][i, :-(-L // c["bs"])].long()
        if fmt == "fp4":
            k, v = (_nearest4(s[x][where].double()).flatten(0, 1)[:L] for x in ("k", "v"))
        else:
            k, v = ((s[x + "c"].view(torch.uint8)[where].view(s[x + "c"].dtype).double() * s[x + "s"][where].double()).flatten(0, 1)[:L]
                    for x in ("k", "v"))
        q = s["q"][at:at + n].double().view(n, c["hkv"], -1, d)
        at += n
        hide = torch.arange(L, device=DEV) > torch.arange(L - n, L, device=DEV).view(n, 1)
        one = []
        for h in range(c["hkv"]):
            def attend(a, b):
                z = torch.einsum("ngd,td->gnt", q[:, h, :, a:b], k[:, h, a:b]) * s["scale"]
                return torch.einsum("gnt,td->ngd", torch.softmax(torch.where(hide, -math.inf, z), -1), v[:, h])

            if c["op"] == "attend4":
                one.append(attend(0, d))
                continue
            lam = s["lambda"].double().view(c["hkv"], -1)[h].view(1, -1, 1)
            y = attend(0, d // 2) - lam * attend(d // 2, d)
            if s["weight"] is not None:
                y = y / ((y * y).mean(-1, keepdim=True) + EPS).sqrt() * s["weight"].double()
            one.append(y * s["out_scale"])
        outs.append(torch.stack(one, 1).reshape(n, c["hq"], d))
    return torch.cat(outs)
