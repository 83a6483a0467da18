"""Oracles of the block tables, the slot map and the writes to the slots.

TEST INFRASTRUCTURE ONLY: plain definitions with Python lists.  Only tests/ and
__graft_entry__.smoke() may use it; the CUDA library never does.
"""

from __future__ import annotations

import numpy as np

ERR_LENGTH, ERR_PAGE, ERR_POOL, ERR_ROWS = 28, 27, 30, 21


def reserve(table, held, lengths, free_pages, free_count, page_size):
    """(table, held, free_pages, free_count, status [B], status of the whole call)."""
    table, held, free = np.array(table), np.array(held), np.array(free_pages)
    B, cols = table.shape
    n = int(free_count)
    status = np.zeros(B, np.int32)
    need = [-(-int(x) // page_size) for x in lengths]
    for b in range(B):
        if not 0 <= held[b] <= cols or lengths[b] < 0 or need[b] > cols:
            status[b] = ERR_LENGTH
    ok = [b for b in range(B) if not status[b]]
    back = sum(max(0, int(held[b]) - need[b]) for b in ok)
    if n < 0 or n + back > len(free):
        return table, held, free, n, status, ERR_POOL
    for b in ok:
        if (table[b, need[b]:held[b]] < 0).any():   # not all of them are pages
            status[b] = ERR_PAGE
    ok = [b for b in ok if not status[b]]
    stack = list(free[:n])
    for b in ok:
        if held[b] > need[b]:
            stack += list(table[b, need[b]:held[b]])
            table[b, need[b]:held[b]] = -1
            held[b] = need[b]
    short = False
    for b in ok:
        want = need[b] - int(held[b])
        if want == 0:
            continue
        short |= want > len(stack)
        if short:
            status[b] = ERR_POOL
            continue
        for c in range(int(held[b]), need[b]):
            table[b, c] = stack.pop()
        held[b] = need[b]
    free[len(stack):n] = -1
    free[:len(stack)] = stack
    return table, held, free, len(stack), status, 0


def slots(table, start, count, rows, page_size):
    """(slots, request, position, offsets, status [B], status of the whole call)."""
    B, cols = table.shape
    take = [max(0, int(c)) for c in count]
    offsets = np.concatenate([[0], np.cumsum(take)]).astype(np.int32)
    out = np.full(rows, -1, np.int64)
    req, pos = np.full(rows, -1, np.int32), np.full(rows, -1, np.int32)
    status = np.zeros(B, np.int32)
    fail = offsets[-1] > rows
    r = 0
    for b in range(B):
        bad = count[b] < 0 or start[b] < 0 or start[b] + count[b] > cols * page_size
        if bad:
            status[b] = ERR_LENGTH
        for i in range(0 if fail else take[b]):
            p = int(start[b]) + i
            req[r], pos[r] = b, (p + 2 ** 31) % 2 ** 32 - 2 ** 31   # as an int32 holds it
            if not bad:
                page = int(table[b, p // page_size])
                if page >= 0:
                    out[r] = page * page_size + p % page_size
                elif not status[b]:
                    status[b] = ERR_PAGE
            r += 1
    return out, req, pos, offsets, status, ERR_ROWS if fail else 0


def write(cache, layer, k, v, where):
    """In place; the first row with a slot outside the pool that is not -1, or -1."""
    pages, _, _, S, _ = cache.shape
    bad = -1
    for r, s in enumerate(where):
        s = int(s)
        if 0 <= s < pages * S:
            cache[s // S, layer, 0, s % S] = k[r].reshape(-1)
            cache[s // S, layer, 1, s % S] = v[r].reshape(-1)
        elif s != -1 and bad < 0:
            bad = r
    return bad
