"""Upkeep of a paged KV cache, request by request on the host (test infrastructure; see
``oracle/__init__``).

The state is a block table, the lengths and a reference count per page. Pages are taken lowest id
first, in request order, then column order. Each function returns new state and the list of
(source, destination) pages to copy; ``None`` stands for "too few free pages".
"""
from __future__ import annotations

import numpy as np


def held(n: int, page_size: int) -> int:
    return -(-int(n) // page_size)


def _free(ref):
    return [p for p in range(len(ref)) if ref[p] == 0]


def resize(table, old, new, ref, page_size):
    table, ref = np.array(table), np.array(ref)
    for r in range(len(old)):
        for j in range(held(new[r], page_size), held(old[r], page_size)):
            ref[table[r, j]] -= 1
            table[r, j] = -1
    want = []
    for r in range(len(old)):
        a, b = held(old[r], page_size), held(new[r], page_size)
        table[r, min(a, b):] = -1
        if new[r] > old[r] and old[r] % page_size and ref[table[r, a - 1]] > 1:
            want.append((r, a - 1, int(table[r, a - 1])))
        want += [(r, j, -1) for j in range(a, b)]
    free = _free(ref)
    if len(free) < len(want):
        return None
    moves = []
    for (r, j, src), page in zip(want, free):
        if src >= 0:
            ref[src] -= 1
            moves.append((src, page))
        table[r, j] = page
        ref[page] = 1
    return table, ref, moves


def fork(table, lens, ref, parents, page_size):
    table, ref = np.array(table), np.array(ref)
    M = table.shape[1]
    for r, n in enumerate(lens):
        for j in range(held(n, page_size)):
            ref[table[r, j]] -= 1
    out = np.full((len(parents), M), -1, dtype=table.dtype)
    out_lens = np.zeros(len(parents), dtype=np.int64)
    seen, want = set(), []
    for r, f in enumerate(parents):
        if f < 0:
            continue
        n = int(lens[f])
        out_lens[r] = n
        h = held(n, page_size)
        out[r, :h] = table[f, :h]
        if n % page_size and f in seen:
            want.append((r, h - 1, int(out[r, h - 1])))
            out[r, h - 1] = -1
        seen.add(f)
        for p in out[r]:
            if p >= 0:
                ref[p] += 1
    free = _free(ref)
    if len(free) < len(want):
        return None
    moves = []
    for (r, j, src), page in zip(want, free):
        out[r, j] = page
        ref[page] = 1
        moves.append((src, page))
    return out, out_lens, ref, moves


def compact(table, ref):
    table, ref = np.array(table), np.array(ref)
    used = [p for p in range(len(ref)) if ref[p] > 0]
    n = len(used)
    page_map = np.full(len(ref), -1, dtype=table.dtype)
    page_map[used] = used
    moves = list(zip([p for p in used if p >= n], [p for p in range(n) if ref[p] == 0]))
    for src, dst in moves:
        page_map[src] = dst
        ref[dst], ref[src] = ref[src], 0
    out = np.where(table >= 0, page_map[np.maximum(table, 0)], -1)
    return out, ref, page_map, moves


def counts(table, lens, num_pages, page_size):
    """The reference counts that a table alone gives."""
    ref = np.zeros(num_pages, dtype=np.int64)
    for r, n in enumerate(lens):
        for j in range(held(n, page_size)):
            ref[table[r][j]] += 1
    return ref
