"""A serving step's metadata and projections, restated from their definitions
(oracle; test infrastructure only).

Planning ([P1] sections 7, 15 and 20): requests own rows of block tables; a
request that brings n new positions takes one block whenever a position
starts one that its row does not hold yet, from the end of the free list, and
each new position's slot is block * block_size + offset.

Norm and rotation: each head's row is divided by the root of its mean square
(plus eps inside the root), multiplied by a gain, and its pairs (a, b) are
turned by the position's angles.
"""

import numpy as np


def plan_step(seq_rows, new_lens, row_lens, row_tables, row_blocks, free_list, block_size, num_tokens):
    """Plan one step, position by position.  row_tables (lists), row_blocks
    and free_list (a stack) are changed in place, as the step's blocks are
    taken.  Returns (block tables as lists, context_lens, query_start,
    positions, slots); None if the free list is too short (then nothing has
    changed)."""
    tables, blocks, stack = [list(t) for t in row_tables], list(row_blocks), list(free_list)
    out_tables, ctx, start, positions, slots = [], [], [0], [], []
    for r, n in zip(seq_rows, new_lens):
        if r < 0:
            out_tables.append([])
            ctx.append(0)
            start.append(start[-1])
            continue
        length = row_lens[r]
        for p in range(length, length + n):
            while p // block_size >= blocks[r]:
                if not stack:
                    return None
                tables[r][blocks[r]] = stack.pop()
                blocks[r] += 1
            positions.append(p)
            slots.append(tables[r][p // block_size] * block_size + p % block_size)
        ctx.append(length + n)
        start.append(start[-1] + n)
        out_tables.append(tables[r][:-(-(length + n) // block_size)])
    assert len(positions) <= num_tokens
    pad = [-1] * (num_tokens - len(positions))
    row_tables[:], row_blocks[:], free_list[:] = tables, blocks, stack
    return out_tables, ctx, start, positions + pad, slots + pad


def release_rows(rows, row_tables, row_blocks, free_list):
    """Give back the rows' blocks, in table order ([P1] section 17)."""
    for r in rows:
        if r >= 0:
            free_list.extend(row_tables[r][:row_blocks[r]])
            row_blocks[r] = 0


def norm_rope(x, gain, eps, position, rot_dim, interleaved, base=10000.0):
    """One head's row x [d] (float64) normed and turned; gain None: no norm."""
    y = np.asarray(x, dtype=np.float64)
    if gain is not None:
        y = y / np.sqrt(np.sum(y * y) / len(y) + eps) * np.asarray(gain, dtype=np.float64)
    y = y.copy()
    half = rot_dim // 2
    for c in range(half):
        angle = position * base ** (-2.0 * c / rot_dim)
        i, j = (2 * c, 2 * c + 1) if interleaved else (c, c + half)
        a, b = y[i], y[j]
        y[i] = a * np.cos(angle) - b * np.sin(angle)
        y[j] = b * np.cos(angle) + a * np.sin(angle)
    return y
