"""Timing cases of the operators around the paged cache.

Five operators, each with its plain form in elementary torch operations
(`own` false) and as calls of this package (`own` true):

  rope     per-head RMS norm of queries and keys and their position rotation
  append   the same with the rotated keys and the values quantized into a pool
  decode   single-token attention over a pool with one scale per block and head
  weights  attention weights of the cached tokens, accumulated over steps
  evict    blocks with the least accumulated weight leave their sequence
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6

# format name -> (the package's constant, bits per element, values of the largest code)
FORMATS = {"fp16": ("KVQ_FP16", 16, 0.0), "int8_token": ("KVQ_INT8_PER_TOKEN", 8, 127.0),
           "int8_group": ("KVQ_INT8_PER_GROUP", 8, 127.0), "e4m3_token": ("KVQ_FP8_E4M3_PER_TOKEN", 8, 448.0),
           "int4_group": ("KVQ_INT4_PER_GROUP", 4, 7.0), "int8_block": ("KVQ_INT8_PER_BLOCK", 8, 127.0),
           "e4m3_block": ("KVQ_FP8_E4M3_PER_BLOCK", 8, 448.0)}


def listed():
    return [
        # one token of each of 8 sequences: a layer's query/key norms and rotation in a decode step (latency)
        {"name": "rope_step", "op": "rope", "T": 8, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "interleaved": False,
         "scaling": "none", "norm": True, "dtype": "bf16"},
        # prompts of 8 x 2048 tokens, half of each head rotated in pairs, positions stretched for a long context
        {"name": "rope_prompt", "op": "rope", "T": 16384, "hq": 32, "hkv": 8, "d": 128, "rot": 64, "interleaved": True,
         "scaling": "parts", "norm": True, "dtype": "fp16"},
        # a decode step's new tokens of 64 sequences into an INT8 per-group pool
        {"name": "append_step", "op": "append", "S": 64, "n": 1, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "scaling": "none", "norm": True, "dtype": "fp16", "fmt": "int8_group", "group": 128, "bs": 16},
        # the same into partly filled blocks with one scale each, whose older codes are rescaled: sequences forked from
        # one prompt, each of which takes its own copy of its last block before it appends to it
        {"name": "append_step_block", "op": "append", "S": 61, "n": 1, "hq": 24, "hkv": 4, "d": 128, "rot": 128,
         "interleaved": True, "scaling": "linear", "norm": False, "dtype": "bf16", "fmt": "int8_block", "group": 0, "bs": 32},
        # prompts of 8 x 2048 tokens into blocks with one scale each
        {"name": "append_prompt", "op": "append", "S": 8, "n": 2048, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "scaling": "bands", "norm": True, "dtype": "bf16", "fmt": "int8_block", "group": 0, "bs": 16},
        # four short requests (latency)
        {"name": "decode_tiny", "op": "decode", "S": 4, "L": 100, "ragged": True, "hq": 4, "hkv": 1, "d": 64,
         "fmt": "int8_block", "bs": 16},
        # the serving batch: 64 sequences of 2048 tokens
        {"name": "decode_batch", "op": "decode", "S": 64, "L": 2048, "ragged": False, "hq": 32, "hkv": 8, "d": 128,
         "fmt": "int8_block", "bs": 16},
        # long contexts in larger blocks, FP8 codes, lengths that differ
        {"name": "decode_long", "op": "decode", "S": 8, "L": 32768, "ragged": True, "hq": 32, "hkv": 8, "d": 128,
         "fmt": "e4m3_block", "bs": 32},
        # the weights of one decode step of the serving batch
        {"name": "weights_batch", "op": "weights", "S": 64, "L": 2048, "ragged": True, "hq": 32, "hkv": 8, "d": 128,
         "fmt": "int8_group", "group": 128, "bs": 16},
        # and of long contexts in blocks with one scale each
        {"name": "weights_long", "op": "weights", "S": 8, "L": 32768, "ragged": False, "hq": 32, "hkv": 8, "d": 128,
         "fmt": "int8_block", "group": 0, "bs": 16},
        # a few short sequences lose a quarter of their blocks
        {"name": "evict_short", "op": "evict", "S": 16, "L": 1000, "ragged": True, "hkv": 8, "bs": 16, "budget": 48,
         "sink": 1, "recent": 4},
        # long contexts cut to an eighth
        {"name": "evict_long", "op": "evict", "S": 8, "L": 32768, "ragged": False, "hkv": 8, "bs": 16, "budget": 256,
         "sink": 4, "recent": 16},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "decode", "decode", "weights", "evict"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 8, 32])
    hq = hkv * (rng.choice([1, 2, 3, 4, 8]) if hkv < 32 else 1)
    turn = {"hq": hq, "hkv": hkv, "d": d, "rot": rng.choice([d, d, d // 2, d // 4]), "interleaved": rng.random() < 0.5,
            "scaling": rng.choice(["none", "linear", "base", "parts", "bands"]), "norm": rng.random() < 0.6,
            "dtype": rng.choice(["fp16", "bf16"])}
    # one 4-bit code more or less is a large step: its borders are for tests, not for these comparisons
    fmt = rng.choice([f for f in FORMATS if op != "append" or f != "int4_group"])
    group = rng.choice([d, d // 2]) if "group" in fmt else 0
    bs = rng.choice([16, 32, 64])
    if op == "rope":
        return {"op": op, "T": _log(rng, 1, 16384 * 40 * 128 // ((hq + hkv) * d)) if (hq + hkv) * d > 40 * 128
                else _log(rng, 1, 16384), **turn}
    if op == "append":
        most = min(16384, 16384 * 48 * 128 // ((hq + 2 * hkv) * d))
        if rng.random() < 0.5:
            return {"op": op, "S": _log(rng, 1, min(256, most)), "n": 1, **turn, "fmt": fmt, "group": group, "bs": bs}
        S = _log(rng, 1, 16)
        return {"op": op, "S": S, "n": _log(rng, 2, max(3, most // S)), **turn, "fmt": fmt, "group": group, "bs": bs}
    if op == "evict":
        S = _log(rng, 1, 64)
        L = _log(rng, 40, min(32768, 8 * 32768 * 8 // (S * hkv)))
        nb = -(-L // bs)
        budget = max(3, int(nb * rng.uniform(0.1, 0.9)))
        sink = rng.randint(0, min(4, budget - 2))
        return {"op": op, "S": S, "L": L, "ragged": rng.random() < 0.7, "hkv": hkv, "bs": bs, "budget": budget,
                "sink": sink, "recent": rng.randint(1, max(1, min(16, budget - sink - 1)))}
    S = _log(rng, 1, 128)
    L = _log(rng, 17, min(32768, 8 * 32768 * 8 * 128 // (S * max(hkv, hq // 4) * d)))
    c = {"op": op, "S": S, "L": L, "ragged": rng.random() < 0.7, "hq": hq, "hkv": hkv, "d": d, "bs": bs}
    if op == "decode":
        return {**c, "fmt": rng.choice(["int8_block", "e4m3_block"])}
    return {**c, "fmt": fmt, "group": group}


def _lens(c):
    """Tokens per sequence: all L, or spread over 1 .. L with the first one L."""
    if not c["ragged"]:
        return [c["L"]] * c["S"]
    return [1 + int((c["L"] - 1) * (1.0 - (s * 0.6180339887498949) % 1.0)) for s in range(c["S"])]


# ------------------------------------------------------------------ work
def _scale_bytes(fmt, group, d, hkv, tokens, blocks):
    if "group" in fmt:
        return tokens * hkv * (d // group) * 4
    if "token" in fmt:
        return tokens * 4
    return blocks * hkv * 4 if "block" in fmt else 0


def work(c):
    op = c["op"]
    if op in ("rope", "append"):
        T = c["T"] if op == "rope" else c["S"] * c["n"]
        q, kv = T * c["hq"] * c["d"], T * c["hkv"] * c["d"]
        per = 6 if c["norm"] else 3
        if op == "rope":
            return {"bytes": 4 * (q + kv) + 8 * T, "flops": per * (q + kv)}
        bits = FORMATS[c["fmt"]][1]
        blocks = c["S"] * -(-c["n"] // c["bs"])
        sc = 2 * _scale_bytes(c["fmt"], c["group"], c["d"], c["hkv"], T, blocks)
        return {"bytes": 4 * q + 4 * kv + 2 * kv * bits // 8 + sc + 16 * T, "flops": per * (q + kv) + 6 * kv}
    lens = _lens(c)
    tokens, blocks = sum(lens), sum(-(-n // c["bs"]) for n in lens)
    if op == "evict":
        kept = sum(min(n, c["budget"] * c["bs"]) for n in lens)
        return {"bytes": 4 * c["hkv"] * (tokens + kept) + 12 * blocks, "flops": tokens * c["hkv"]}
    codes = tokens * c["hkv"] * c["d"] * FORMATS[c["fmt"]][1] // 8  # K, or V
    sc = _scale_bytes(c["fmt"], c.get("group", 0), c["d"], c["hkv"], tokens, blocks)
    rows = c["S"] * c["hq"]
    if op == "decode":
        return {"bytes": 2 * (codes + sc) + rows * c["d"] * 6 + 4 * blocks, "flops": 4 * tokens * c["hq"] * c["d"]}
    return {"bytes": codes + sc + rows * (2 * c["d"] + 4) + 8 * tokens * c["hkv"] + 4 * blocks,
            "flops": 2 * tokens * c["hq"] * c["d"]}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _rope_config(c):
    """The rotation's settings as the package's kvq_rope_init takes them."""
    factor = {"none": 1.0, "linear": 4.0, "base": 8.0, "parts": 16.0, "bands": 8.0}[c["scaling"]]
    lo, hi = {"parts": (1.0, 32.0), "bands": (1.0, 4.0)}.get(c["scaling"], (0.0, 0.0))
    return {"base": 10000.0 if c["scaling"] != "bands" else 500000.0, "factor": factor, "orig_len": 8192.0, "low": lo, "high": hi}


def _frequencies(c):
    """Radians per position of each pair, and the factor on cos and sin."""
    r, f = c["rot"], _rope_config(c)
    i = np.arange(r // 2, dtype=np.float64)
    base, s, n = f["base"], f["factor"], f["orig_len"]
    if c["scaling"] == "base":
        base = base * s ** (r / (r - 2.0))
    w = base ** (-2.0 * i / r)
    m = 1.0
    if c["scaling"] == "linear":
        w = w / s
    elif c["scaling"] == "parts":
        edge = [r * math.log(n / (2 * math.pi * b)) / (2 * math.log(base)) for b in (f["high"], f["low"])]
        lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), r - 1)
        ramp = np.clip((i - lo) / ((hi - lo) or 0.001), 0.0, 1.0)
        w = w / s * ramp + w * (1.0 - ramp)
        m = 0.1 * math.log(s) + 1.0
    elif c["scaling"] == "bands":
        turns = n * w / (2 * math.pi)
        mix = np.clip((turns - f["low"]) / (f["high"] - f["low"]), 0.0, 1.0)
        w = (1.0 - mix) * w / s + mix * w
    return torch.from_numpy(w).to(DEV), m


def _rows(c, T, seed):
    """A layer's projected rows [T][q heads | k heads | v heads], the norms' weights and the tokens' positions."""
    g = _gen(seed)
    dt = torch.float16 if c["dtype"] == "fp16" else torch.bfloat16
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    gain = 1.0 + 9.0 * (torch.rand((hq + 2 * hkv) * d, generator=g, device=DEV) < 0.01)
    qkv = (_randn(g, T, (hq + 2 * hkv) * d) * gain).to(dt).view(T, hq + 2 * hkv, d)
    s = {"q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:],
         "positions": torch.randint(0, 131072, (T,), generator=g, device=DEV), "q_weight": None, "k_weight": None}
    if c["norm"]:
        s["q_weight"], s["k_weight"] = 1.0 + 0.1 * _randn(g, d), 1.0 + 0.1 * _randn(g, d)
    return s


def _slots(c, seed):
    """Where a call's tokens go: slots [S*n], the touched blocks' token rows `at` [blocks][bs] (-1: none of this call)
    and how many older tokens each block holds."""
    S, n, bs = c["S"], c["n"], c["bs"]
    r = np.random.RandomState(seed % (1 << 31))
    if n == 1:
        first = (7 * np.arange(S) + 3) % bs  # a decode step: the tokens land all over their blocks
    else:
        first = np.zeros(S, np.int64)
    per = (n + bs - 1) // bs if n > 1 else 1
    blocks = r.permutation(S * per + 3)[:S * per].reshape(S, per)
    t = first[:, None] + np.arange(n)
    slots = np.take_along_axis(blocks, t // bs, 1) * bs + t % bs
    at = np.full((S, per * bs), -1, np.int64)
    np.put_along_axis(at, t, np.arange(S * n).reshape(S, n), 1)
    old = np.where(np.arange(per) == 0, first[:, None], 0).reshape(-1)
    return slots.reshape(-1), blocks.reshape(-1), at.reshape(S * per, bs), old, S * per + 3


def _as_fp8(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _div(a, b):
    """IEEE a / b with zeros where b is zero (a divisor that is a plain number may be multiplied by instead)."""
    return torch.where(b == 0, torch.zeros_like(a), a / torch.where(b == 0, torch.ones_like(b), b))


def _scale(amax, top):
    return amax / torch.full((), top, device=DEV, dtype=amax.dtype)


def _codes(x, s, fmt):
    """Codes of x at scale s, as the numbers they stand for before the scale."""
    y = _div(x, s.expand_as(x))
    if "e4m3" in fmt:
        return _as_fp8(y).to(x.dtype)
    top = FORMATS[fmt][2]
    return y.round().clamp(-top, top)


def _quantize(x, fmt, group):
    """(codes, scales) of tokens x [T, H, D], or of blocks x [N, bs, H, D] where the format has a scale per block."""
    top = FORMATS[fmt][2]
    if "block" in fmt:
        s = _scale(x.abs().amax((1, 3), keepdim=True), top)
    elif "token" in fmt:
        s = _scale(x.abs().amax((-2, -1), keepdim=True), top)
    else:
        x = x.unflatten(-1, (-1, group))
        s = _scale(x.abs().amax(-1, keepdim=True), top)
    c = _codes(x, s, fmt)
    return (c, s) if "group" not in fmt else (c.flatten(-2), s.expand_as(c).flatten(-2))


def _cache(c, seed):
    """A filled cache: fp16 tokens K, V [N, bs, H, D], their codes and scales, the block table and the lengths."""
    g = _gen(seed)
    S, hkv, d, bs, fmt = c["S"], c["hkv"], c["d"], c["bs"], c["fmt"]
    lens = _lens(c)
    nb = -(-c["L"] // bs)
    N = S * nb
    gain = 1.0 + 9.0 * (torch.rand(hkv * d, generator=g, device=DEV) < 0.01)
    perm = torch.randperm(N, generator=g, device=DEV).to(torch.int32)
    s = {"table": perm.view(S, nb), "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
         "q": _randn(g, S, c["hq"], d).half(), "scale": d ** -0.5, "blocks": N}
    at = torch.arange(nb * bs, device=DEV).view(1, nb, bs)
    filled = torch.zeros((N, bs), dtype=torch.bool, device=DEV)
    filled[perm.long()] = (at < s["lens"].view(S, 1, 1)).view(N, bs)
    for x in ("k", "v"):
        t = (_randn(g, N, bs, hkv * d) * gain).half().view(N, bs, hkv, d) * filled.view(N, bs, 1, 1)
        s[x] = t
        if fmt == "fp16":
            s[x + "c"], s[x + "s"] = t, None
            continue
        codes, sc = _quantize(t.float(), fmt, c.get("group", 0))
        s[x + "c"] = _as_fp8(codes) if "e4m3" in fmt else codes.to(torch.int8)
        s[x + "s"] = sc[..., ::c["group"]].contiguous() if "group" in fmt else sc
    s["filled"] = filled
    return s


def _values(s, x, c, dtype):
    """The cache of x ("k" or "v") along each sequence, in `dtype`: [S, tokens, H, D]."""
    code, sc = s[x + "c"], s[x + "s"]
    at = s["table"].long()
    if code.dtype == torch.float8_e4m3fn:
        y = code.view(torch.uint8)[at].view(torch.float8_e4m3fn).to(dtype)
    else:
        y = code[at].to(dtype)
    if sc is not None:
        t = sc[at].to(dtype)
        y = (y.unflatten(-1, (t.shape[-1], -1)) * t.unsqueeze(-1)).flatten(-2) if "group" in c["fmt"] else y * t
    return y.flatten(1, 2)


def _logits(s, c, dtype):
    """q . k * scale along each sequence, [S, H, group of heads, tokens], -inf behind its length."""
    k = _values(s, "k", c, dtype)
    q = s["q"].to(dtype).unflatten(1, (c["hkv"], -1))
    z = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    past = torch.arange(z.shape[-1], device=DEV) >= s["lens"].view(-1, 1, 1, 1)
    return z.masked_fill(past, -math.inf)


def _fill_pool(s, c):
    """The package's pool with the same tokens."""
    import paged_quantized_kv_kvq_gb300 as kvq

    pool = kvq.KVPool(s["blocks"], c["bs"], c["hkv"], c["d"], getattr(kvq, FORMATS[c["fmt"]][0]), c.get("group", 0), device=DEV)
    slots = torch.arange(s["blocks"] * c["bs"], device=DEV)
    slots = torch.where(s["filled"].view(-1), slots, -1)
    pool.append(s["k"].flatten(0, 1), s["v"].flatten(0, 1), slots)
    return pool


def prepare(c, seed):
    op = c["op"]
    if op in ("rope", "append"):
        T = c["T"] if op == "rope" else c["S"] * c["n"]
        s = _rows(c, T, seed)
        s["case"] = c
        s["w"], s["m"] = _frequencies(c)
        if own:
            import paged_quantized_kv_kvq_gb300 as kvq

            s["kvq"] = kvq
            s["plan"] = kvq.kvq_rope_init(c["rot"], interleaved=c["interleaved"], scaling=getattr(kvq, "KVQ_ROPE_" + c["scaling"].upper()),
                                          **_rope_config(c))
            s["q_out"] = torch.empty((T, c["hq"], c["d"]), dtype=torch.float16, device=DEV)
            s["k_out"] = torch.empty((T, c["hkv"], c["d"]), dtype=torch.float16, device=DEV)
        if op == "rope":
            return s
        slots, blocks, at, old, num = _slots(c, seed)
        s["at"] = torch.from_numpy(at).to(DEV)
        s["old"] = torch.from_numpy(old).to(DEV)
        s["slots"] = torch.from_numpy(slots).to(DEV)
        if "block" in c["fmt"]:  # what the call leaves in every block it touches, older tokens among it
            o = np.arange(c["bs"])
            rows = (at >= 0) | (o < old[:, None])
            s["read"] = torch.from_numpy((blocks[:, None] * c["bs"] + o)[rows]).to(DEV)
            s["rows"] = torch.from_numpy(rows).to(DEV)
            s["before"] = None
            if c["n"] == 1:
                g = _gen(seed + 7)
                b = (0.5 * _randn(g, 2, len(blocks), c["bs"], c["hkv"], c["d"])).half()
                s["before"] = b * (torch.arange(c["bs"], device=DEV) < s["old"].view(-1, 1)).view(1, -1, c["bs"], 1, 1)
                s["before_codes"], s["before_scales"] = _quantize(s["before"].float().flatten(0, 1), c["fmt"], 0)
        else:
            s["read"] = s["slots"]
        if own:
            # a block that grows takes its scale with it, so the older tokens stay in blocks of their own, which every
            # pass copies: appending to the same blocks once more would find their scales grown already
            forks = "block" in c["fmt"] and s["before"] is not None
            s["pool"] = kvq.KVPool(2 * num if forks else num, c["bs"], c["hkv"], c["d"], getattr(kvq, FORMATS[c["fmt"]][0]),
                                   c["group"], device=DEV)
            if forks:
                o = np.arange(c["bs"])
                was = np.where(o < old[:, None], (num + blocks[:, None]) * c["bs"] + o, -1).reshape(-1)
                s["pool"].append(s["before"][0].flatten(0, 1), s["before"][1].flatten(0, 1), torch.from_numpy(was).to(DEV))
                s["to"] = torch.from_numpy(blocks.astype(np.int32)).to(DEV)
                s["from"] = s["to"] + num
            n = s["read"].numel()
            s["k_values"] = torch.empty((n, c["hkv"], c["d"]), dtype=torch.float16, device=DEV)
            s["v_values"] = torch.empty_like(s["k_values"])
        return s
    if op == "evict":
        g = _gen(seed)
        lens = _lens(c)
        nb = -(-c["L"] // c["bs"])
        s = {"case": c, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
        # accumulated weights: a few heavy blocks over a long tail
        heavy = (1.5 * _randn(g, c["S"], 1, nb)).repeat_interleave(c["bs"], 2)[..., :c["L"]]
        s["scores"] = torch.exp(heavy + _randn(g, c["S"], c["hkv"], c["L"])) / c["L"]
        s["table"] = torch.randperm(c["S"] * nb, generator=g, device=DEV).to(torch.int32).view(c["S"], nb)
        if own:
            import paged_quantized_kv_kvq_gb300 as kvq

            s["kvq"] = kvq
            s["pool"] = kvq.KVPool(1, c["bs"], c["hkv"], 64, kvq.KVQ_FP16, device=DEV)
            s["table_out"] = torch.empty_like(s["table"])
            s["lens_out"] = torch.empty_like(s["lens"])
            s["kept"] = torch.empty((c["S"], c["budget"]), dtype=torch.int32, device=DEV)
            s["scores_out"] = torch.zeros((c["S"], c["hkv"], c["budget"] * c["bs"]), device=DEV)
        return s
    s = _cache(c, seed)
    s["case"] = c
    if op == "weights":
        g = _gen(seed + 7)
        s["lse"] = torch.logsumexp(_logits(s, c, torch.float64), -1).float().flatten(1)
        s["prev"] = torch.rand((c["S"], c["hkv"], c["L"]), generator=g, device=DEV) / c["L"]
        s["prev"] *= torch.arange(c["L"], device=DEV) < s["lens"].view(-1, 1, 1)
        s["decay"] = 0.95
    if own:
        import paged_quantized_kv_kvq_gb300 as kvq

        s["kvq"], s["pool"] = kvq, _fill_pool(s, c)
        if op == "decode":
            ws = kvq.kvq_decode_workspace_bytes(s["pool"].handle, c["S"], c["hq"], c["L"])
            s["ws"] = torch.empty(max(ws, 1), dtype=torch.uint8, device=DEV)
            s["out"] = torch.empty((c["S"], c["hq"], c["d"]), device=DEV)
        else:
            s["scores"] = torch.zeros_like(s["prev"])
    for x in ("k", "v"):  # the fp16 tokens themselves are no part of the cache
        if c["fmt"] != "fp16" or own:
            del s[x]
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    c, kvq = s["case"], s["kvq"]
    if c["op"] == "rope":
        kvq.kvq_rope(s["plan"], s["q"], s["k"], s["positions"], s["q_out"], s["k_out"], s["q_weight"], s["k_weight"], EPS)
        return {"q": s["q_out"], "k": s["k_out"]}
    h = s["pool"].handle
    if c["op"] == "append":
        if "from" in s:
            kvq.kvq_copy_blocks(h, s["from"], s["to"])
        kvq.kvq_rope_append(h, s["plan"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_out"], s["q_weight"],
                            s["k_weight"], EPS)
        kvq.kvq_read_values(h, s["read"], s["k_values"], s["v_values"])
        return {"q": s["q_out"], "k": s["k_values"], "v": s["v_values"]}
    if c["op"] == "decode":
        kvq.kvq_paged_decode(h, s["q"], s["table"], s["lens"], c["L"], s["scale"], s["out"], s["ws"])
        return s["out"]
    if c["op"] == "weights":
        kvq.kvq_attention_weights(h, s["q"], s["table"], s["lens"], c["L"], s["scale"], s["lse"], s["scores"], s["prev"], s["decay"])
        return s["scores"]
    kvq.kvq_evict_blocks(h, s["scores"], s["table"], s["lens"], c["L"], c["budget"], c["sink"], c["recent"], s["table_out"],
                         s["lens_out"], s["kept"], s["scores_out"])
    return {"table": s["table_out"], "lens": s["lens_out"], "kept": s["kept"], "scores": s["scores_out"]}


def _turned(s, x, weight):
    """Norm and rotation of rows x, in 32 bits; the angles in 64."""
    c = s["case"]
    r, x = c["rot"], x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    a = s["positions"].double().unsqueeze(1) * s["w"]
    cos, sin = (torch.cos(a) * s["m"]).float().unsqueeze(1), (torch.sin(a) * s["m"]).float().unsqueeze(1)
    if c["interleaved"]:
        u, v = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((u * cos - v * sin, u * sin + v * cos), -1).flatten(-2)
    else:
        u, v = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((u * cos - v * sin, u * sin + v * cos), -1)
    return torch.cat((y, x[..., r:]), -1)


def _stored(s, x, side):
    """What the cache holds of the call's tokens x [T, H, D] (and, with a scale per block, of the blocks' older ones)."""
    c = s["case"]
    fmt = c["fmt"]
    if fmt == "fp16":
        return x.half()
    if "block" not in fmt:
        codes, sc = _quantize(x, fmt, c["group"])
        return (codes * sc).half()
    new = s["at"] >= 0
    y = torch.where(new.view(*new.shape, 1, 1), x[s["at"].clamp(min=0)], 0.0)
    sc = _scale(y.abs().amax((1, 3), keepdim=True), FORMATS[fmt][2])
    codes = None
    if s["before"] is not None:
        n = len(s["at"])
        was = s["before_scales"][side * n:(side + 1) * n]
        old = s["before_codes"][side * n:(side + 1) * n]
        was = torch.where((s["old"] > 0).view(-1, 1, 1, 1), was, 0.0)
        sc = torch.maximum(sc, was)
        codes = torch.where(sc > was, _codes(old * was, sc, fmt), old)
    put = _codes(y, sc, fmt)
    codes = put if codes is None else torch.where(new.view(*new.shape, 1, 1), put, codes)
    return (codes * sc)[s["rows"]].half()


def _plain(s):
    c = s["case"]
    if c["op"] == "rope":
        return {"q": _turned(s, s["q"], s["q_weight"]).half(), "k": _turned(s, s["k"], s["k_weight"]).half()}
    if c["op"] == "append":
        return {"q": _turned(s, s["q"], s["q_weight"]).half(), "k": _stored(s, _turned(s, s["k"], s["k_weight"]), 0),
                "v": _stored(s, s["v"].float(), 1)}
    if c["op"] == "evict":
        return _plain_evict(s)
    z = _logits(s, c, torch.float32)
    if c["op"] == "decode":
        p = torch.exp(z - z.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        return torch.matmul(p, _values(s, "v", c, torch.float32).transpose(1, 2)).flatten(1, 2)
    w = torch.exp(z[..., :c["L"]] - s["lse"].unflatten(1, (c["hkv"], -1)).unsqueeze(-1)).sum(2)
    return s["decay"] * s["prev"] + w


def _plain_evict(s):
    c = s["case"]
    S, bs, L, budget = c["S"], c["bs"], c["L"], c["budget"]
    nb = s["table"].shape[1]
    inside = torch.arange(L, device=DEV) < s["lens"].view(-1, 1, 1)
    w = torch.zeros((S, c["hkv"], nb * bs), device=DEV)
    w[..., :L] = torch.where(inside, s["scores"], 0.0)
    w = w.view(S, c["hkv"], nb, bs)
    b = w.double().sum((1, 3)).float()  # next to the border 32-bit sums would decide by their order
    j = torch.arange(nb, device=DEV)
    n = ((s["lens"] + bs - 1) // bs).view(-1, 1)
    held = (j < c["sink"]) | (j >= n - c["recent"])
    b = torch.where(held, math.inf, b).masked_fill(j >= n, -math.inf)
    order = torch.sort(b, dim=1, descending=True, stable=True).indices
    rank = torch.zeros_like(order).scatter_(1, order, j.expand(S, nb))
    keep = (rank < budget) & (j < n)
    # kept blocks in their order, then the evicted ones, then what lies behind the sequence
    first = torch.where(keep, j, torch.where(j < n, j + nb, j + 2 * nb))
    at = torch.sort(first, dim=1).indices
    count = keep.sum(1, keepdim=True)
    kept = torch.full((S, max(budget, nb)), -1, device=DEV, dtype=torch.int64)
    kept[:, :nb] = torch.where(j < count, at, -1)
    kept = kept[:, :budget]
    lens = s["lens"] - ((n - count) * bs).view(-1).to(torch.int32)
    out = torch.take_along_dim(w, kept.clamp(min=0).view(S, 1, budget, 1), 2).flatten(2)
    out = torch.where(torch.arange(budget * bs, device=DEV) < lens.view(-1, 1, 1), out, 0.0)
    return {"table": torch.take_along_dim(s["table"], at, 1), "lens": lens, "kept": kept.to(torch.int32), "scores": out}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(c, seed):
    op = c["op"]
    if op in ("rope", "append"):
        T = c["T"] if op == "rope" else c["S"] * c["n"]
        s = _rows(c, T, seed)
        w, m = _frequencies(c)
        angle = s["positions"].to(torch.float64)[:, None, None] * w
        rotor = torch.polar(torch.full_like(angle, m), angle)

        def turned(x, weight):
            x = x.double()
            if weight is not None:
                x = x / ((x * x).mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
            y = x.clone()
            r = c["rot"]
            u = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) if c["interleaved"] else \
                torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous())
            u = u * rotor
            if c["interleaved"]:
                y[..., 0:r:2], y[..., 1:r:2] = u.real, u.imag
            else:
                y[..., :r // 2], y[..., r // 2:r] = u.real, u.imag
            return y

        q, k = turned(s["q"], s["q_weight"]), turned(s["k"], s["k_weight"])
        if op == "rope":
            return {"q": q, "k": k}
        return {"q": q, "k": _exact_stored(c, seed, k, 0), "v": _exact_stored(c, seed, s["v"].double(), 1)}
    if op == "evict":
        return _exact_evict(c, seed)
    s = _cache(c, seed)
    outs = []
    lens = _lens(c)
    lse = prev = None
    if op == "weights":
        p = prepare(c, seed)
        lse, prev = p["lse"].double(), p["prev"].double()
    for i, n in enumerate(lens):  # one sequence after the other: 64 bits of a long one fill some memory
        one = {"table": s["table"][i:i + 1]}
        one |= {x + y: s[x + y] for x in ("k", "v") for y in ("c", "s")}
        k = _values(one, "k", c, torch.float64)[0, :n]
        q = s["q"][i].double().view(c["hkv"], -1, c["d"])
        z = torch.einsum("hgd,thd->hgt", q, k) * s["scale"]
        if op == "decode":
            v = _values(one, "v", c, torch.float64)[0, :n]
            outs.append(torch.einsum("hgt,thd->hgd", torch.softmax(z, -1), v).reshape(c["hq"], c["d"]))
        else:
            y = torch.zeros((c["hkv"], c["L"]), dtype=torch.float64, device=DEV)
            y[:, :n] = 0.95 * prev[i, :, :n] + torch.exp(z - lse[i].view(c["hkv"], -1, 1)).sum(1)
            outs.append(y)
    return torch.stack(outs)


def _exact_stored(c, seed, x, side):
    """The values of the touched tokens by the format's definition, in 64 bits; a stored scale has 32."""
    fmt, bs, d = c["fmt"], c["bs"], c["d"]
    if fmt == "fp16":
        return x
    top = torch.full((), FORMATS[fmt][2], dtype=torch.float64, device=DEV)

    def nearest(y, s):
        y = y / torch.where(s == 0, torch.ones_like(s), s)
        return (_as_fp8(y.float()).double() if "e4m3" in fmt else torch.round(y).clamp(-top, top)) * s

    if "block" not in fmt:
        y = x.reshape(len(x), -1, c["group"]) if "group" in fmt else x.reshape(len(x), 1, -1)
        return nearest(y, (y.abs().amax(-1, keepdim=True) / top).float().double()).view_as(x)
    p = prepare(c, seed)
    at, old = p["at"], p["old"]
    new = at >= 0
    y = torch.where(new[:, :, None, None], x[at.clamp(min=0)], 0.0)
    s = (y.abs().amax((1, 3), keepdim=True) / top).float().double()
    before = torch.zeros_like(y)
    if p["before"] is not None:
        n = len(at)
        codes, was = (p[z][side * n:(side + 1) * n].double() for z in ("before_codes", "before_scales"))
        was = torch.where(old[:, None, None, None] > 0, was, 0.0)
        grown = torch.maximum(s, was)
        before = torch.where(grown > was, nearest(codes * was, grown), codes * was)
        s = grown
    return torch.where(new[:, :, None, None], nearest(y, s), before)[p["rows"]]


def _exact_evict(c, seed):
    p = prepare(c, seed)
    w, table, bs = p["scores"].double().cpu().numpy(), p["table"].cpu().numpy(), c["bs"]
    tables, kepts = table.copy(), np.full((c["S"], c["budget"]), -1, np.int32)
    lens_out, out = np.zeros(c["S"], np.int32), np.zeros((c["S"], c["hkv"], c["budget"] * bs))
    for i, L in enumerate(_lens(c)):
        n = -(-L // bs)
        must = [j for j in range(n) if j < c["sink"] or j >= n - c["recent"]]
        sums = [np.float32(w[i, :, j * bs:min(L, (j + 1) * bs)].sum()) for j in range(n)]
        free = sorted((j for j in range(n) if j not in set(must)), key=lambda j: (-sums[j], j))
        kept = sorted(must + free[:max(0, c["budget"] - len(must))])
        gone = [j for j in range(n) if j not in set(kept)]
        tables[i, :n] = table[i, kept + gone]
        kepts[i, :len(kept)] = kept
        lens_out[i] = L - len(gone) * bs
        for a, j in enumerate(kept):
            m = min(L - j * bs, bs)
            out[i, :, a * bs:a * bs + m] = w[i, :, j * bs:j * bs + m]
    return {"table": torch.from_numpy(tables), "lens": torch.from_numpy(lens_out), "kept": torch.from_numpy(kepts),
            "scores": torch.from_numpy(out)}
