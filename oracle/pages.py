"""A step's pages, request by request over a free list (oracle; test only).

The free list is a stack. Blocks given back (by requests whose length falls) are put aside in the
order of their requests; growing requests take from them first, then from the stack; what is left
goes onto the stack, the last first. Placement is that of ``metadata``: position p lives on rank
``(p // S) % W`` in block ``local_index // block_size`` ("Context Parallel Guide (PCP & DCP)",
"How it works" items 1 and 2).
"""

from __future__ import annotations

import numpy as np

from . import metadata as _md

STATUS_BAD_PAGE = 0x8
STATUS_HELD_BACK = 0x80


def plan(*, targets, seq_lens, block_table, free_list, free_count, max_rows, dcp, interleave, block_size,
         max_local_len, num_blocks, rank_begin=0, num_ranks=None):
    nr = dcp - rank_begin if num_ranks is None else num_ranks
    table = np.array(block_table, dtype=np.int64)
    stack_room = np.array(free_list, dtype=np.int64)
    status = 0
    if not 0 <= free_count <= num_blocks:
        status |= STATUS_BAD_PAGE
        free_count = min(max(free_count, 0), num_blocks)

    def local(n):  # rank 0 holds the most
        return _md.local_len_closed_form(n, 0, dcp, interleave)

    def blocks(n):
        return -(-local(n) // block_size)

    old, new = [int(x) for x in seq_lens], [int(x) for x in targets]
    lens = list(old)
    aside, growing = [], []
    for b, (a, t) in enumerate(zip(old, new)):
        if a < 0 or t < 0:
            status |= _md.STATUS_BAD_SEQ_LEN
        elif local(max(a, t)) > max_local_len:
            status |= _md.STATUS_LOCAL_OVER_BOUND
        elif t > a:
            growing.append(b)
        else:
            aside += [int(x) for x in table[b, blocks(t): blocks(a)]]
            lens[b] = t
    stack = [int(x) for x in stack_room[:free_count]]
    rows = need = taken = 0
    at = {}
    for b in growing:
        rows += new[b] - old[b]
        need += blocks(new[b]) - blocks(old[b])
        if rows > max_rows or need > len(aside) + free_count:
            status |= STATUS_HELD_BACK
            break
        for i in range(blocks(old[b]), blocks(new[b])):
            table[b, i] = aside[taken] if taken < len(aside) else stack.pop()
            taken += 1
            if not 0 <= table[b, i] < num_blocks:
                status |= _md.STATUS_BAD_BLOCK_ID
        lens[b] = new[b]
        at[b] = True
    for x in reversed(aside[taken:]):
        if len(stack) < num_blocks:
            if not 0 <= x < num_blocks:
                status |= _md.STATUS_BAD_BLOCK_ID
            stack_room[len(stack)] = x
            stack.append(x)
        else:
            status |= STATUS_BAD_PAGE
    slots = np.full((nr, max_rows), -1, dtype=np.int64)
    positions = np.zeros(max_rows, dtype=np.int64)
    cu, row = [0], 0
    for b in range(len(old)):
        if b in at:
            for p in range(old[b], new[b]):
                positions[row] = p
                k = int(_md.owner(p, dcp, interleave)) - rank_begin
                li = int(_md.local_index(p, dcp, interleave))
                block = int(table[b, li // block_size])
                if not 0 <= block < num_blocks:
                    status |= _md.STATUS_BAD_BLOCK_ID
                elif 0 <= k < nr:
                    slots[k, row] = block * block_size + li % block_size
                row += 1
        cu.append(row)
    return dict(new_lens=np.array(lens), block_table=table, free_list=stack_room, free_count=len(stack),
                slot_mapping=slots, positions=positions, cu_rows=np.array(cu), status=status)
