"""Block tables grown and shrunk over a stack of free blocks, one request, one
token at a time.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""

import numpy as np


def extend(table, past, new, free, count, block_size, max_tokens, num_blocks):
    """(table, context_lens, q_starts, slots, positions, block_starts, count,
    lacking, good) of giving request b new[b] tokens behind its past[b]; `good`
    is false where something was refused or a block id was bad; `lacking` is -1
    where the whole step was, with no block missing."""
    table = table.copy()
    B, MB = table.shape
    good, plan = True, []
    for b in range(B):
        p, n = int(past[b]), int(new[b])
        if p < 0 or n < 0 or p + n > MB * block_size:
            good, n = False, 0
        have = -(-p // block_size)
        plan.append((p, n, have, -(-(p + n) // block_size) - have))
    need = sum(x[3] for x in plan)
    tokens = sum(x[1] for x in plan)
    in_range = 0 <= count <= len(free)
    lacking = max(0, need - count) if in_range else need
    goes = in_range and need <= count and tokens <= max_tokens
    lacking = -1 if not goes and not lacking else lacking
    good = good and in_range and tokens <= max_tokens
    slots = np.full(max_tokens, -1, dtype=np.int64)
    positions = np.full(max_tokens, -1, dtype=np.int64)
    ctx, q_starts, block_starts = np.array(past, dtype=np.int32), [0], [0]
    t = 0
    for b, (p, n, have, k) in enumerate(plan):
        if goes:
            for i in range(k):
                count -= 1
                ok = 0 <= free[count] < num_blocks
                good = good and ok
                table[b, have + i] = free[count] if ok else -1
            for pos in range(p, p + n):
                blk = table[b, pos // block_size]
                ok = 0 <= blk < num_blocks
                good = good and ok
                slots[t] = int(blk) * block_size + pos % block_size if ok else -1
                positions[t] = pos
                t += 1
            ctx[b] = p + n
            q_starts.append(q_starts[-1] + n)
            block_starts.append(block_starts[-1] + k)
        else:
            q_starts.append(0)
            block_starts.append(0)
    return (table, ctx, np.array(q_starts, dtype=np.int32), slots, positions, np.array(block_starts, dtype=np.int32),
            count, lacking, good)


def truncate(table, ctx, keep, free, count, block_size, num_blocks):
    """(free, count, good) after request b gave back what lies behind its first keep[b] tokens."""
    free = free.copy()
    MB = table.shape[1]
    good, back = True, []
    for b in range(len(ctx)):
        c, k = int(ctx[b]), int(keep[b])
        if k < 0 or k > c or c > MB * block_size:
            good = False
            continue
        back += [int(table[b, j]) for j in range(-(-k // block_size), -(-c // block_size))]
    if count < 0 or count + len(back) > len(free):
        return free, count, False
    for blk in reversed(back):                        # the last taken goes back first
        ok = 0 <= blk < num_blocks
        good = good and ok
        free[count] = blk if ok else -1
        count += 1
    return free, count, good
