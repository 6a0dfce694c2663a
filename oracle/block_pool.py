"""Oracle: block tables, slot mappings and the block pool as plain loops (test
infrastructure; see the package docstring).

"Quantized KV caches in production", PagedAttention: a sequence's blocks are
found through its table; slot = block * block_size + offset.  The pages give
no allocator: the order (rows ascending when blocks are taken, descending when
they are given back) is the library's stated contract.
"""
from __future__ import annotations

import numpy as np

BLOCK = 16


class Pool:
    """free: stack of block ids (the last goes next); refs: rows that use each block."""

    def __init__(self, free, num_blocks):
        self.free = [int(x) for x in free]
        self.refs = np.zeros(num_blocks, dtype=np.int64)


def assign_blocks(pool, new_lens, context_lens, tables, max_tokens, prefix_rows=None, prefix_blocks=None):
    """Updates context_lens, tables and pool in place; returns (ok, offsets,
    slots, positions).  Nothing changes unless all of it can be done."""
    rows, width = tables.shape
    c0 = [int(c) for c in context_lens]
    start = list(c0)
    ok = all(int(n) >= 0 for n in new_lens) and all(c >= 0 for c in c0)
    for r in range(rows):
        s = -1 if prefix_rows is None else int(prefix_rows[r])
        if s >= 0:
            k = int(prefix_blocks[r])
            if s >= rows or s == r or c0[r] != 0 or k < 0 or k > width or k * BLOCK > c0[s]:
                ok = False
            else:
                start[r] = k * BLOCK
    need = 0
    for r in range(rows):
        n = int(new_lens[r])
        if not ok:
            break
        if start[r] + n > width * BLOCK:
            ok = False
        elif n > 0 and start[r] % BLOCK:
            last = int(tables[r, start[r] // BLOCK])
            if not 0 <= last < len(pool.refs) or pool.refs[last] != 1:
                ok = False
        need += -(-(start[r] + n) // BLOCK) - -(-start[r] // BLOCK)
    blocks = range(len(pool.refs))
    for r in range(rows):
        if ok and prefix_rows is not None and prefix_rows[r] >= 0:  # blocks that it would share
            ok = all(int(x) in blocks for x in tables[prefix_rows[r], :start[r] // BLOCK])
    if ok and need <= len(pool.free):                                # blocks that it would take
        ok = all(x in blocks for x in pool.free[len(pool.free) - need:])
    if not ok or need > len(pool.free) or sum(int(n) for n in new_lens) > max_tokens:
        return False, np.zeros(rows + 1, np.int32), np.full(max_tokens, -1, np.int64), np.full(max_tokens, -1, np.int32)
    offsets, slots, positions = [0], [], []
    for r in range(rows):
        if prefix_rows is not None and prefix_rows[r] >= 0:
            for i in range(start[r] // BLOCK):
                tables[r, i] = tables[prefix_rows[r], i]
                pool.refs[tables[r, i]] += 1
        for p in range(start[r], start[r] + int(new_lens[r])):
            if p % BLOCK == 0:
                tables[r, p // BLOCK] = pool.free.pop()
                pool.refs[tables[r, p // BLOCK]] = 1
            slots.append(int(tables[r, p // BLOCK]) * BLOCK + p % BLOCK)
            positions.append(p)
        context_lens[r] = start[r] + int(new_lens[r])
        offsets.append(len(slots))
    pad = [-1] * (max_tokens - len(slots))
    return True, np.array(offsets, np.int32), np.array(slots + pad, np.int64), np.array(positions + pad, np.int32)


def release_blocks(pool, keep_lens, context_lens, tables):
    """Rows keep their first keep_lens tokens; updated in place."""
    rows, width = tables.shape
    for r in reversed(range(rows)):
        keep, c = int(keep_lens[r]), int(context_lens[r])
        if keep < 0 or c < 0 or c > width * BLOCK or keep >= c:
            continue
        for i in reversed(range(-(-keep // BLOCK), -(-c // BLOCK))):
            block = int(tables[r, i])
            tables[r, i] = -1
            if not 0 <= block < len(pool.refs) or pool.refs[block] < 1:
                continue
            pool.refs[block] -= 1
            if pool.refs[block] == 0:
                pool.free.append(block)
        context_lens[r] = keep
