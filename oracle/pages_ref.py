"""Block tables, slot maps and rows at slots (test infrastructure only).

"投机解码的树状注意力验证：一次前向如何并行校验多条候选路径", section
"实现中的 KV Cache 与批处理约束": a paged cache frees and reuses pages around every
step; "02 · Token Tree 与 Tree Attention" §4: pages of rejected nodes are reclaimed.
The readings: the list of free pages is a stack, requests are served in their
order, and what cannot be served is refused from the first request on that does
not fit.
"""

import numpy as np

ST_BAD_SIZE, ST_BAD_BLOCK, ST_NO_BLOCKS = 1, 8, 128
PAGE = 16


def block_tables_ref(want, table, n_blocks, free, num_blocks, status, released=None, released_count=None):
    """One call on plain lists: table[b] holds max_blocks entries, free is the
    stack (last entry on top). Returns the new (table, n_blocks, free, status,
    released_count); nothing of the arguments is changed."""
    table = [list(r) for r in table]
    n, free, status = list(n_blocks), list(free), list(status)
    count = [0] * len(n) if released_count is None else list(released_count)
    width = len(table[0]) if table else 0
    need = [-(-w // PAGE) for w in want]
    inside = lambda ids: all(0 <= i < num_blocks for i in ids)
    flag, on = [0] * len(n), []
    for b in range(len(n)):
        if status[b]:
            continue
        if want[b] < 0 or need[b] > width or not 0 <= n[b] <= width or not 0 <= count[b] <= width:
            flag[b] = ST_BAD_SIZE
        else:
            on.append(b)
    total = sum(count[b] + max(n[b] - need[b], 0) for b in on)
    if len(free) + total > num_blocks:
        return table, n, free, [s or ST_BAD_SIZE for s in status], count
    for b in list(on):
        back = table[b][need[b]:n[b]] + (list(released[b][:count[b]]) if count[b] else [])
        if not inside(back):
            flag[b] = ST_BAD_BLOCK
            on.remove(b)
    for b in reversed(on):
        free += reversed(released[b][:count[b]] if count[b] else [])
    for b in reversed(on):
        free += reversed(table[b][need[b]:n[b]])
    out = False
    for b in on:
        count[b] = 0
        if n[b] > need[b]:
            table[b][need[b]:n[b]] = [-1] * (n[b] - need[b])
            n[b] = need[b]
        elif n[b] < need[b]:
            out = out or need[b] - n[b] > len(free)
            if out:
                flag[b] = ST_NO_BLOCKS
                continue
            while n[b] < need[b]:
                table[b][n[b]] = free.pop()
                n[b] += 1
    return table, n, free, [s | f for s, f in zip(status, flag)], count


def slot_map_ref(cu, start, table, n_blocks, num_blocks, rows, status):
    """(slots, status) of a ragged batch's rows."""
    slots, status = np.full(rows, -1, np.int64), list(status)
    high = None
    for b in range(len(start)):
        c0, c1 = int(cu[b]), int(cu[b + 1])
        high = c0 if high is None else max(high, c0)
        if c1 == c0 or status[b]:
            continue
        if c1 < c0 or c0 < high or c0 < 0 or c1 > rows or start[b] < 0:
            status[b] |= ST_BAD_SIZE
            continue
        s = int(start[b]) + np.arange(c1 - c0)
        pages = s // PAGE
        if pages[-1] >= min(int(n_blocks[b]), len(table[b])):
            status[b] |= ST_BAD_BLOCK
            continue
        ids = np.asarray(table[b], np.int64)[pages]
        if (ids < 0).any() or (ids >= num_blocks).any():
            status[b] |= ST_BAD_BLOCK
            continue
        slots[c0:c1] = ids * PAGE + s % PAGE
    return slots, status
