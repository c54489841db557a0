"""Where a step's new tokens go (include/pkv.h, pkv_plan_step), sequence by sequence.
Test infrastructure: only tests and the smoke check use it.

The rules are the page pool's (Notebook 10, section 5): blocks are added when a sequence
crosses a block boundary, counted before any is taken, and come off the top of the free
stack in sequence order.
"""

from __future__ import annotations

import numpy as np

BLOCK = 16


def plan(lens, new, held, free, left, tables, num_rows, num_blocks=1 << 31):
    """Returns dict(slots, positions, start, lens, held, left, result, tables, bad)."""
    batch, width = tables.shape
    tables = tables.copy()
    bad = False
    counts = []
    for n, m, h in zip(lens, new, held):
        n, m, h = int(n), int(m), int(h)
        fine = n >= 0 and m >= 0 and 0 <= h <= width and n <= BLOCK * h and n + m <= BLOCK * width
        bad |= not fine
        counts.append((m, max(-(-(n + m) // BLOCK) - h, 0)) if fine else (0, 0))
    rows, need = sum(m for m, _ in counts), sum(k for _, k in counts)
    slots, positions = np.full(num_rows, -1, np.int64), np.full(num_rows, -1, np.int32)
    count_ok = 0 <= left <= len(free)
    bad |= not count_ok or rows > num_rows
    out = dict(slots=slots, positions=positions, start=np.zeros(batch + 1, np.int32), lens=np.array(lens, np.int32),
               held=np.array(held, np.int32), left=int(left), tables=tables,
               result=[0, max(need - left, 0) if count_ok else 0])
    if count_ok and rows <= num_rows and need <= left:
        stack = [int(b) for b in free[:left]]
        r = 0
        for i, (m, k) in enumerate(counts):
            out["start"][i] = r
            for b in range(k):
                block = stack.pop()
                fine = 0 <= block < num_blocks
                bad |= not fine
                tables[i, int(held[i]) + b] = block if fine else -1
            for t in range(int(lens[i]), int(lens[i]) + m):
                block = int(tables[i, t // BLOCK])
                if 0 <= block < num_blocks:
                    slots[r] = block * BLOCK + t % BLOCK
                else:
                    bad = True
                positions[r] = t
                r += 1
            out["lens"][i] += m
            out["held"][i] += k
        out["start"][batch] = r
        out["left"], out["result"] = len(stack), [rows, 0]
    out["bad"] = bool(bad)
    return out
