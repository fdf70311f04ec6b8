"""Plain reference of a step's block bookkeeping, for the tests: one sequence after the
other, one token after the other."""
from __future__ import annotations

import numpy as np


def _ceil(a, b):
    return -(-a // b)


def release(table, old, new, free, count, bs, num_blocks, shared=0):
    """(free list, count, error) after the blocks beyond `new` tokens came back."""
    free, err = np.array(free), False
    if not 0 <= count <= len(free):
        count, err = min(max(count, 0), len(free)), True
    width = table.shape[1]
    for s in range(len(old)):
        a, b = int(old[s]), int(new[s])
        err |= a < 0 or b < 0 or _ceil(max(a, 0), bs) > width
        for j in range(max(_ceil(max(b, 0), bs), shared), min(_ceil(max(a, 0), bs), width)):
            i = int(table[s, j])
            if not 0 <= i < num_blocks or count == len(free):
                err = True
                continue
            free[count] = i
            count += 1
    return free, count, err


def extend(n, table, lens, free, count, bs, num_blocks, max_tokens):
    """dict of the call's outputs, and whether it reports an error."""
    table, lens = np.array(table), np.array(lens, np.int64)
    slots, pos = np.full(max_tokens, -1, np.int64), np.zeros(max_tokens, np.int64)
    q_start, err = [0], False
    if not 0 <= count <= len(free):
        count, err = min(max(count, 0), len(free)), True
    row = wanted = taken = 0
    for s in range(len(n)):
        L, k = int(lens[s]), int(n[s])
        fits = L >= 0 and k >= 0 and L + k <= table.shape[1] * bs
        need = _ceil(L + k, bs) - _ceil(L, bs) if fits else 0
        wanted += need
        served = fits and row + k <= max_tokens and (need == 0 or wanted <= count)
        if served:
            for j in range(need):
                i = int(free[count - 1 - taken])
                taken += 1
                table[s, _ceil(L, bs) + j] = i
                err |= not 0 <= i < num_blocks
        else:
            err = True
        for i in range(max(k, 0)):
            p = max(L, 0) + i
            if row + i < max_tokens:
                pos[row + i] = p
                if served:
                    b = int(table[s, p // bs])
                    if 0 <= b < num_blocks:
                        slots[row + i] = b * bs + p % bs
                    else:
                        err = True
        row = min(row + max(k, 0), max_tokens)
        q_start.append(row)
        if served:
            lens[s] = L + k
    return {"table": table, "lens": lens.astype(np.int32), "count": count - taken, "q_start": np.array(q_start, np.int32),
            "slots": slots, "positions": pos}, err
