"""Plain statements of the drafted step's operators (numpy, CPU).

Test infrastructure only, written from the formulas: one request and one node
after another.  Attention is ``cache_oracle.attention`` over what a node sees.
"""
from __future__ import annotations

import numpy as np

PAGE = 64


def ancestors(parent):
    """For every node the set of its ancestors and itself; None for a node whose parent is not an earlier one."""
    sets = []
    for i, p in enumerate(parent):
        ok = -1 <= p < i
        sets.append(((sets[p] or set()) if p >= 0 else set()) | {i} if ok else None)
    return sets


def chain(n):
    return [i - 1 for i in range(n)]


def plan(length, count, parent, token, table, num_pages, rows, max_nodes, words):
    """(req_start, positions, cache_pos, mask, row_token) of a drafted step."""
    max_pages = table.shape[1]
    start = [0]
    positions, cache_pos = np.zeros(rows, int), np.full(rows, -1)
    mask, row_token = np.zeros((rows, words), np.uint32), np.zeros(rows, int)
    for r, (at, n) in enumerate(zip(length, count)):
        if not (0 <= n <= max_nodes and at >= 0 and at + n <= PAGE * max_pages):
            n = 0
        n = min(n, rows - start[-1])
        up = chain(n) if parent is None else [int(p) for p in parent[r][:n]]
        for i, seen in enumerate(ancestors(up)):
            t = start[-1] + i
            positions[t] = at + len(seen or {0}) - 1
            page = table[r, (at + i) // PAGE]
            if seen is not None and 0 <= page < num_pages:
                cache_pos[t] = at + i
            for j in seen or ():
                mask[t, j // 32] |= np.uint32(1 << (j % 32))
            row_token[t] = token[r][i] if token is not None else 0
        start.append(start[-1] + n)
    return np.array(start), positions, cache_pos, mask, row_token


def sees(length, n, i, mask_row, num_pages, table_row):
    """The positions that node i of a request with n nodes reads (mask_row None: a chain)."""
    nodes = range(i + 1) if mask_row is None else [
        j for j in range(min(n, 32 * len(mask_row))) if (int(mask_row[j // 32]) >> (j % 32)) & 1]
    return [s for s in [*range(length), *(length + j for j in nodes)] if 0 <= table_row[s // PAGE] < num_pages]


def accept(start, length, parent, row_token, target, cache_pos, max_nodes):
    """(path, accepted, next, new_len): children by hand, the lowest first."""
    path, accepted, after, new_len = np.full((len(length), max_nodes), -1), [], [], []
    for r, at in enumerate(length):
        t0, n = start[r], start[r + 1] - start[r]
        up = chain(n) if parent is None else [int(p) for p in parent[r][:n]]
        stored = [cache_pos is None or cache_pos[t0 + i] >= 0 for i in range(n)]
        taken = [0] if n > 0 and stored[0] else []
        while taken:
            p = taken[-1]
            fits = [i for i in range(p + 1, n) if up[i] == p and stored[i] and row_token[t0 + i] == target[t0 + p]]
            if not fits:
                break
            taken.append(fits[0])
        path[r, :len(taken)] = taken
        accepted.append(len(taken))
        after.append(int(target[t0 + taken[-1]]) if taken else -1)
        new_len.append(at + len(taken))
    return path, accepted, after, new_len


def move(pool, row_bytes, scale_bytes, table, length, path, count):
    """uint8 pool [pages, heads, bytes] after the moves, from a copy of what was there."""
    was, out = pool.copy(), pool.copy()
    for r, at in enumerate(length):
        for d in range(count[r]):
            src, dst = at + path[r][d], at + d
            a, b = table[r, src // PAGE], table[r, dst // PAGE]
            if not (0 <= a < len(pool) and 0 <= b < len(pool)):
                continue
            x, y, base = src % PAGE, dst % PAGE, PAGE * row_bytes
            out[b, :, y * row_bytes:(y + 1) * row_bytes] = was[a, :, x * row_bytes:(x + 1) * row_bytes]
            out[b, :, base + y * scale_bytes:base + (y + 1) * scale_bytes] = (
                was[a, :, base + x * scale_bytes:base + (x + 1) * scale_bytes])
    return out


def trim(table, ref, old, new):
    """The page table and the reference counts with every request's end released."""
    table, ref = table.copy(), ref.copy()
    for r in range(len(old)):
        for j in range(-(-new[r] // PAGE), -(-old[r] // PAGE)):
            if table[r, j] >= 0:
                ref[table[r, j]] -= 1
            table[r, j] = -1
    return table, ref
