"""ORACLE -- test infrastructure only (tests).

Reference for the page tables (the pages of the sources have no counterpart), one request and
one page at a time, as the definition in include/hpa.h states it.
"""
from __future__ import annotations

PAGE = 64
BAD_SEQLEN, BAD_PAGE, OVERFLOW, BAD_MAP, NO_PAGES = 1, 4, 16, 32, 128


def assign(seq_lens, new_tokens, table, held, free, num_pages, rows=None, pos_offset=None,
           max_tokens=None):
    """One step on plain lists: table [num_rows][stride], held [num_rows], free (the stack, bottom
    first, its top last).  Returns (state after: table, held, free), (indptr, indices), (slots,
    positions), status; entries of the table past a row's count are those of before."""
    table, held, free = [list(x) for x in table], list(held), list(free)
    B, stride, status = len(seq_lens), len(table[0]), 0
    rows = list(range(B)) if rows is None else list(rows)
    new = [0] * B if new_tokens is None else list(new_tokens)
    good, seen = [], set()
    for r in range(B):
        bad = 0
        if not 0 <= rows[r] < len(table) or rows[r] in seen:
            bad |= BAD_MAP
            rows[r] = -1
        elif not 0 <= held[rows[r]] <= stride:
            bad |= BAD_MAP
            seen.add(rows[r])
            rows[r] = -1
        if rows[r] >= 0:
            seen.add(rows[r])
        if seq_lens[r] < 0 or new[r] < 0 or new[r] > seq_lens[r]:
            bad |= BAD_SEQLEN
        if -(-max(seq_lens[r], 0) // PAGE) > stride:
            bad |= OVERFLOW
        status |= bad
        good.append(not bad)
    need = [-(-seq_lens[r] // PAGE) if good[r] else None for r in range(B)]
    for r in range(B):                               # pages go back
        if good[r]:
            row = table[rows[r]]
            for i in range(need[r], held[rows[r]]):
                free.append(row[i])
            held[rows[r]] = min(held[rows[r]], need[r])
    empty = False
    for r in range(B):                               # and come off the stack
        if not good[r] or need[r] <= held[rows[r]]:
            continue
        if empty or need[r] - held[rows[r]] > len(free):
            empty, good[r], status = True, False, status | NO_PAGES
            continue
        while held[rows[r]] < need[r]:
            table[rows[r]][held[rows[r]]] = free.pop()
            held[rows[r]] += 1
    indptr, indices, slots, positions = [0], [], [], []
    for r in range(B):
        if rows[r] >= 0:
            indices += table[rows[r]][:held[rows[r]]]
        indptr.append(len(indices))
        for j in range(max(new[r], 0)):
            pos = max(seq_lens[r] - new[r] + j, 0)
            slots.append(table[rows[r]][pos // PAGE] * PAGE + pos % PAGE if good[r] else -1)
            positions.append(pos + (0 if pos_offset is None else pos_offset[r]))
    if max_tokens is not None:
        if len(slots) > max_tokens:
            status |= OVERFLOW
        pad = max(0, max_tokens - len(slots))
        slots = (slots + [-1] * pad)[:max_tokens]
        positions = (positions + [0] * pad)[:max_tokens]
    return (table, held, free), (indptr, indices), (slots, positions), status
