"""Block tables, slot map and positions from request lengths, on the CPU.

Page 2 §4.3 and page 3: the cache is paged and a block table maps a request's
positions to blocks; page 2 §3.3: what lies past the accepted prefix is
dropped.  The pages do not say how blocks are handed out.  Readings taken:

* free block ids stand in a ring: ids are taken from its head and returned to
  its tail, both in (request, page) order; what a call returns is free from
  the next call on;
* a request holds the pages of all its positions, or, with a window, those of
  the sinks and of the positions that its first new row can still see;
* a request gets its pages if the ring holds what it and every request before
  it ask for; else it takes none and does not run;
* length -1 means that the request has ended;
* a ring or table entry that is no block id (a corrupt state) serves no row and
  is given to nobody: the request that takes it (the table then holds -1) or
  would write to it does not run (its rows are -1, it keeps its pages), and what
  is returned to the ring are block ids alone.

Written page by page with sets; no interval arithmetic.
"""
from __future__ import annotations

import numpy as np

CAPACITY, INVALID, BOUNDS = 2, 1, 6


def oracle_block_tables(ctx_lens, row_start, parent, rows, block_table, span, pool, pool_state,
                        slots, positions, M, window=0, sinks=0, block=16):
    """Returns a dict of the arrays after the call and the status bits raised;
    inputs are not modified."""
    B, max_blocks = block_table.shape
    nb = len(pool)
    table, sp, ring = block_table.copy(), span.copy(), pool.copy()
    slots, positions = slots.copy(), positions.copy()
    ok = np.zeros(B, dtype=np.int32)
    head, count = int(pool_state[0]), int(pool_state[1])
    status = 0
    pool_ok = 0 <= head < nb and 0 <= count <= nb
    if not pool_ok:
        status |= 1 << BOUNDS
    sink_pages = -(-sinks // block) if window else 0
    rows_ok = row_start is None or bool(
        np.all(np.diff(row_start) >= 0) and row_start[0] >= 0 and row_start[B] <= rows)
    if not rows_ok:  # every row is none's
        slots[:rows], positions[:rows] = -1, -1

    def pages(lo, hi):
        return {p for p in range(hi) if p < sink_pages or p >= lo}

    asked, taken, returned = 0, 0, []
    new_state = []
    for b in range(B):
        ctx = int(ctx_lens[b])
        if row_start is None:
            r0, r1 = b * M, b * M + M
        else:
            r0, r1 = int(row_start[b]), int(row_start[b + 1])
        lo, hi = int(sp[b, 0]), int(sp[b, 1])
        code = None
        if not pool_ok or not 0 <= lo <= hi <= max_blocks:
            code = BOUNDS
        elif ctx < -1 or not rows_ok:
            code = INVALID
        elif parent is not None and ctx >= 0 and (
                parent[b, 0] != -1 or any(not 0 <= parent[b, n] < n for n in range(1, M))):
            code = INVALID
        elif ctx >= 0 and ctx + r1 - r0 > max_blocks * block:
            code = CAPACITY
        lo2 = max(0, ctx - window + 1) // block if window and ctx >= 0 else 0
        if code is None and ctx >= 0 and hi > 0 and lo2 < lo:
            code = INVALID
        served = code is None and ctx >= 0
        held = pages(lo, hi) if code is None else set()
        want = set()
        hi2 = 0
        if served:
            hi2 = -(-(ctx + r1 - r0) // block)
            want = pages(lo2, hi2)
            need = sorted(want - held)
            asked += len(need)
            if need and asked > count:
                status |= 1 << CAPACITY
                served = False
                hi2 = min(hi, hi2)
                lo2 = min(lo2, hi2)
            else:
                for p in need:
                    table[b, p] = ring[(head + taken) % nb]
                    taken += 1
                    if not 0 <= table[b, p] < nb:
                        table[b, p] = -1
                        status |= 1 << BOUNDS
                        served = False
                for t in range(ctx, ctx + r1 - r0):
                    if not 0 <= table[b, t // block] < nb:
                        status |= 1 << BOUNDS
                        served = False
        if code is not None:
            status |= 1 << code
        else:
            for p in sorted(held - want):
                returned.append(int(block_table[b, p]))
                table[b, p] = -1
            new_state.append((b, lo2, hi2))
        ok[b] = served
        for r in range(r0, r1) if rows_ok else ():
            slots[r], positions[r] = -1, -1
            if served:
                i = r - r0
                t = ctx + i
                slots[r] = int(table[b, t // block]) * block + t % block
                depth, n = 0, i
                while parent is not None and n > 0:
                    n, depth = int(parent[b, n]), depth + 1
                positions[r] = ctx + (i if parent is None else depth)
    for b, lo2, hi2 in new_state:
        sp[b] = lo2, hi2
    back = [i for i in returned if 0 <= i < nb]
    if len(back) < len(returned):
        status |= 1 << BOUNDS
    for j in range(len(returned)):
        ring[(head + count + j) % nb] = back[j] if j < len(back) else -1
    state = np.array([(head + taken) % nb, count - taken + len(back)], dtype=np.int32)
    if not pool_ok:
        state = np.array(pool_state, dtype=np.int32)
    return dict(block_table=table, span=sp, pool=ring, pool_state=state, slots=slots,
                positions=positions, ok=ok, status=status)
