"""Binary64 oracle of attention over a paged cache and of the cache's pages.

TEST INFRASTRUCTURE ONLY, like the rest of this package: a sequence, a head and a page at a time, from the definitions, sharing
nothing with the HIP library.
"""
from __future__ import annotations

import math
from dataclasses import dataclass
from typing import List, Optional, Sequence, Tuple

import numpy as np

STATUS_OK = 0
STATUS_BAD_PAGE = 7
STATUS_BAD_LENGTH = 8
STATUS_BAD_PARENT = 9
STATUS_NO_PAGE = 10


@dataclass
class AttendRow:
    """One sequence: out [q_heads, dim], lse [q_heads], weights [q_heads, slots], and what an error bound is made of."""
    status: int
    out: np.ndarray
    lse: np.ndarray
    weights: np.ndarray
    scores: Optional[np.ndarray] = None       # [q_heads, n] unscaled
    magnitude: Optional[np.ndarray] = None    # [q_heads, n] sum |q_i k_i|
    values: Optional[np.ndarray] = None       # [kv_heads, n, dim]


def attend_row(q, k_pages, v_pages, table_row, length: int, scale: float, window: int = 0, weights_slots: int = 0) -> AttendRow:
    """q [q_heads, dim]; pages [pages, kv_heads, slots, dim]; all as binary64 arrays of the stored values."""
    hq, dim = q.shape
    pages, hk, slots, _ = k_pages.shape
    nan = AttendRow(STATUS_BAD_LENGTH, np.full((hq, dim), np.nan), np.full(hq, np.nan), np.full((hq, weights_slots), np.nan))
    if length < 0 or length > len(table_row) * slots or (weights_slots and length > weights_slots):
        return nan
    lo = max(0, length - window) if window else 0
    where = [(int(table_row[j // slots]), j % slots) for j in range(lo, length)]
    if any(p < 0 or p >= pages for p, _ in where):
        nan.status = STATUS_BAD_PAGE
        return nan
    r = AttendRow(STATUS_OK, np.zeros((hq, dim)), np.full(hq, -np.inf), np.zeros((hq, weights_slots)))
    if not where:
        return r
    pg, sl = np.array([p for p, _ in where]), np.array([s for _, s in where])
    r.scores, r.magnitude = np.zeros((hq, len(where))), np.zeros((hq, len(where)))
    r.values = np.stack([v_pages[pg, h, sl] for h in range(hk)])
    for h in range(hq):
        kv = h // (hq // hk)
        keys = k_pages[pg, kv, sl]
        with np.errstate(invalid="ignore"):
            r.scores[h] = (keys * q[h]).sum(1)
            r.magnitude[h] = np.abs(keys * q[h]).sum(1)
        m = r.scores[h].max()
        if m == -np.inf:
            continue
        with np.errstate(invalid="ignore"):
            e = np.exp(scale * (r.scores[h] - m))
        total = math.fsum(e) if np.isfinite(e).all() else np.nan
        w = e / total
        r.lse[h] = scale * m + math.log(total)
        with np.errstate(invalid="ignore"):
            r.out[h] = w @ r.values[kv]
        if weights_slots:
            r.weights[h, lo:length] = w
    return r


def append(lengths, offsets, table, slots: int, pages: int, tokens: int) -> Tuple[List[Tuple[int, int, int]], List[int]]:
    """(token, page, slot) of every token that is written, and each sequence's status."""
    moves, status = [], []
    for b, n in enumerate(lengths):
        start, end = int(offsets[b]), int(offsets[b + 1])
        if not (0 <= start <= end <= tokens) or n < end - start or n > len(table[b]) * slots:
            status.append(STATUS_BAD_LENGTH)
            continue
        st = STATUS_OK
        for t in range(start, end):
            j = n - (end - t)
            p = int(table[b][j // slots])
            if 0 <= p < pages:
                moves.append((t, p, j % slots))
            else:
                st = STATUS_BAD_PAGE
        status.append(st)
    return moves, status


@dataclass
class ForkResult:
    table: List[List[int]]
    lengths: List[int]
    refs: List[int]
    status: List[int]
    copies: List[Tuple[int, int]]     # (page, page that receives its contents)


def fork(table, lengths, refs: Sequence[int], parent, n_new, slots: int, width: int) -> ForkResult:
    """The definition, a sequence and a page at a time."""
    refs, pages = [int(x) for x in refs], len(refs)
    held, bad = [], []
    for row, n in zip(table, lengths):
        ok = 0 <= n <= len(row) * slots
        used = [int(p) for p in row[: -(-n // slots)]] if ok else []
        st = STATUS_BAD_LENGTH if not ok else STATUS_BAD_PAGE if any(p < 0 or p >= pages for p in used) else STATUS_OK
        held.append(used)
        bad.append(st)
    room = width * slots
    first = {}
    plan = []       # per child: status, inherited length, whether its last page is copied
    for i, p in enumerate(parent):
        if p < -1 or p >= len(lengths):
            plan.append([STATUS_BAD_PARENT, 0, False, -1])
        elif p == -1:
            plan.append([STATUS_OK, 0, False, -1])
        elif bad[p] != STATUS_OK:
            plan.append([bad[p], 0, False, -1])
        elif lengths[p] > room:
            plan.append([STATUS_BAD_LENGTH, 0, False, -1])
        else:
            plan.append([STATUS_OK, lengths[p], p in first and lengths[p] % slots != 0, p])
            first.setdefault(p, i)
    # all sequences let go of their pages, all children take hold of what they share
    for s, used in enumerate(held):
        if bad[s] == STATUS_OK:
            for page in used:
                refs[page] -= 1
    for status, n, copied, p in plan:
        if p >= 0:
            for page in held[p][: len(held[p]) - int(copied)]:
                refs[page] += 1
    free = [p for p in range(pages) if refs[p] <= 0]
    out, taken, give_back = ForkResult([], [], refs, [], []), 0, []
    for (status, n, copied, p), grow in zip(plan, n_new):
        total = n
        if status == STATUS_OK:
            if grow < 0 or n + grow > room:
                status = STATUS_BAD_LENGTH
            else:
                total = n + grow
        need = int(copied) + -(-total // slots) - -(-n // slots)
        row = list(held[p]) if p >= 0 else []
        found = need == 0 or taken + need <= len(free)      # who needs no page misses none, whoever came before
        if found:
            fresh = free[taken: taken + need]
            if copied:
                out.copies.append((row[-1], fresh[0]))
                row[-1] = fresh[0]
                fresh = fresh[1:]
            row += fresh
        else:
            status = status if status != STATUS_OK else STATUS_NO_PAGE
            total = n
            if copied:
                give_back += row[:-1]
                row, total = [], 0
        for page in free[taken: taken + need] if found else []:
            refs[page] = 1
        taken += need
        out.table.append(row + [-1] * (width - len(row)))
        out.lengths.append(total)
        out.status.append(status)
    for page in give_back:
        refs[page] -= 1
    return out


@dataclass
class CompactResult:
    table: List[List[int]]
    refs: List[int]
    map: List[int]
    count: int
    status: List[int]
    moves: List[Tuple[int, int]]


def compact(table, lengths, refs, slots: int) -> CompactResult:
    refs = [int(x) for x in refs]
    live = [p for p, r in enumerate(refs) if r > 0]
    n = len(live)
    holes = [p for p in range(n) if refs[p] <= 0]
    moves = list(zip([p for p in live if p >= n], holes))
    to = [-1] * len(refs)
    for p in live:
        to[p] = p
    for src, dst in moves:
        to[src] = dst
    out_refs = [0] * len(refs)
    for p in live:
        out_refs[to[p]] = refs[p]
    rows, status = [], []
    for row, length in zip(table, lengths):
        if length < 0 or length > len(row) * slots:
            rows.append([int(p) for p in row])
            status.append(STATUS_BAD_LENGTH)
            continue
        used, st, out = -(-length // slots), STATUS_OK, []
        for x, p in enumerate(row):
            p = int(p)
            if x >= used:
                out.append(-1)
            elif 0 <= p < len(refs) and to[p] >= 0:
                out.append(to[p])
            else:
                out.append(p)
                st = STATUS_BAD_PAGE
        rows.append(out)
        status.append(st)
    return CompactResult(rows, out_refs, to, n, status, moves)


def copy_pairs(source, target, pages: int) -> Tuple[List[Tuple[int, int]], List[int]]:
    """The copies that are made, and every pair's status. Of the sound pairs with one target the last is copied."""
    targets, last, status = list(map(int, target)), {}, []
    for i, (s, t) in enumerate(zip(map(int, source), targets)):
        bad = not (0 <= s < pages and 0 <= t < pages) or any(x == s for j, x in enumerate(targets) if j != i)
        status.append(STATUS_BAD_PAGE if bad else STATUS_OK)
        if not bad:
            last[t] = i
    return [(int(source[i]), targets[i]) for i in sorted(last.values())], status
