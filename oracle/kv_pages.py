"""CPU oracle of the cache's page operators and of the tree path commit
(include/spec_kv_pages.h).

TEST INFRASTRUCTURE, like the rest of ``oracle/``.  Plain serial loops over
sequences, columns and pages; every function updates its arrays in place and
returns the set of error names met.
"""
from __future__ import annotations

import numpy as np


def _columns(n: int, page_size: int) -> int:
    return -(-n // page_size)


def release(new_len, seq_len, table, ref, page_size: int):
    errors = set()
    for b in range(table.shape[0]):
        to = int(seq_len[b]) if new_len is None else int(new_len[b])
        if new_len is not None and to < 0:
            continue
        if seq_len[b] < 0 or to > seq_len[b]:
            errors.add("LENGTH")
            continue
        cols = [c for c in range(_columns(to, page_size), table.shape[1]) if table[b, c] >= 0]
        bad = {"PAGE" for c in cols if table[b, c] >= len(ref)}
        bad |= {"REF" for c in cols if table[b, c] < len(ref) and ref[table[b, c]] < 1}
        if bad:
            errors |= bad
            continue
        for c in cols:
            ref[table[b, c]] -= 1
            table[b, c] = -1
        seq_len[b] = to
    return errors


def fork(src, dst, seq_len, table, ref, page_size: int):
    errors = set()
    B, cols = table.shape
    for i, (s, d) in enumerate(zip(src.tolist(), dst.tolist())):
        if not (0 <= s < B and 0 <= d < B) or s == d or d in dst[:i].tolist() or s in dst.tolist():
            errors.add("PAIR")
            continue
        if seq_len[s] < 0:
            errors.add("LENGTH")
            continue
        used = _columns(int(seq_len[s]), page_size)
        if used > cols:
            errors.add("CAPACITY")
            continue
        bad = {"BUSY"} if (table[d] >= 0).any() else set()
        for p in table[s, :used].tolist():
            if not 0 <= p < len(ref):
                bad.add("PAGE")
            elif ref[p] < 1:
                bad.add("REF")
        if bad:
            errors |= bad
            continue
        table[d] = -1
        table[d, :used] = table[s, :used]
        for p in table[s, :used].tolist():
            ref[p] += 1
        seq_len[d] = seq_len[s]
    return errors


def reserve(num_new, seq_len, table, ref, pool, page_size: int):
    """All or nothing; as if the sequences were served in order."""
    errors, served = set(), []
    for b in range(table.shape[0]):
        n, L = int(num_new[b]), int(seq_len[b])
        if n == 0:
            continue
        if n < 0 or L < 0:
            errors.add("LENGTH")
            continue
        first, last = L // page_size, (L + n - 1) // page_size
        if last >= table.shape[1]:
            errors.add("CAPACITY")
            continue
        bad = set()
        for c in range(first, last + 1):
            p = int(table[b, c])
            if p >= len(ref) or (p < 0 and c == first and L % page_size):
                bad.add("PAGE")
            elif p >= 0 and ref[p] < 1:
                bad.add("REF")
        if bad:
            errors |= bad
        else:
            served.append((b, L, first, last))
    t, r, moves = table.copy(), ref.copy(), []
    free = [p for p in range(len(ref)) if ref[p] <= 0]
    for b, L, first, last in served:
        for c in range(first, last + 1):
            p = int(t[b, c])
            if p >= 0 and r[p] <= 1:
                continue
            if not free:
                return errors | {"POOL"}
            q = free.pop(0)
            if p >= 0:
                r[p] -= 1
                if c == first and L % page_size:
                    moves.append((p, q, L % page_size))
            t[b, c], r[q] = q, 1
    for p, q, n in moves:
        pool[:, q, :n] = pool[:, p, :n]
    table[:], ref[:] = t, r
    return errors


def compact(table, ref, pool):
    """Returns (errors, live pages)."""
    errors = {"REF"} if (ref < 0).any() else set()
    live = int((ref > 0).sum())
    holes = [p for p in range(live) if ref[p] <= 0]
    movers = [p for p in range(live, len(ref)) if ref[p] > 0]
    to = dict(zip(movers, holes))
    for b in range(table.shape[0]):
        for c in range(table.shape[1]):
            p = int(table[b, c])
            if p < 0:
                continue
            if p < len(ref) and ref[p] > 0:
                table[b, c] = to.get(p, p)
            else:
                errors.add("PAGE")
    for p, q in to.items():
        pool[:, q] = pool[:, p]
        ref[q], ref[p] = ref[p], 0
    return errors, live


def commit_path(num_accepted, path, seq_len, table, pool, staged, page_size: int):
    errors = set()
    B, N = path.shape

    def spot(b, pos):
        c = pos // page_size
        if c >= table.shape[1]:
            errors.add("CAPACITY")
            return None
        p = int(table[b, c])
        if not 0 <= p < pool.shape[1]:
            errors.add("PAGE")
            return None
        return p, pos % page_size

    for b in range(B):
        n, L = int(num_accepted[b]), int(seq_len[b])
        if L < 0:
            errors.add("LENGTH")
            continue
        if n < 0:
            continue
        nodes = [0] + path[b, :min(n, N)].tolist()
        if n >= N or any(y <= x or y >= N for x, y in zip(nodes, nodes[1:])):
            errors.add("PATH")
            continue
        to = [spot(b, L + i) for i in range(n + 1)]
        come = [(b, x) if staged is not None else spot(b, L + x) for x in nodes]
        if None in to or None in come:
            continue
        held = [np.array(staged[:, b, x] if staged is not None else pool[:, come[i][0], come[i][1]])
                for i, x in enumerate(nodes)]
        for i in range(n + 1):
            pool[:, to[i][0], to[i][1]] = held[i]
        seq_len[b] = L + n + 1
    return errors
