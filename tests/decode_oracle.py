"""The operators of a decoding step, written from their definitions in 64 bits with numpy,
one row or request at a time.  They share no code with the library."""
import math

import numpy as np


def sample_row(x, u, t, top_k=None, top_p=None, min_p=None):
    """(token, log-probability, margin): margin is the distance, relative to the kept
    weight, of u's place from the nearest running sum (how far rounding may move it)."""
    x = np.asarray(x, dtype=np.float64).copy()
    x[np.isnan(x)] = -np.inf
    if x.size == 0 or x.max() == -np.inf:
        return -1, -math.inf, 1.0
    top = x.max()
    if not t > 0:
        return int(np.flatnonzero(x == top)[0]), 0.0, 1.0
    with np.errstate(invalid="ignore", over="ignore", divide="ignore", under="ignore"):
        y = np.where(x == top, 0.0, (x - top) / np.float64(t))
        w = np.where(x == -np.inf, 0.0, np.exp(y))
    order = np.lexsort((np.arange(x.size), -x))
    keep = x.size
    if top_k is not None and top_k > 0:
        keep = min(keep, int(top_k))
    if top_p is not None and not top_p >= 1:
        p = float(top_p) if top_p > 0 else 0.0
        sums = np.cumsum(w[order[:keep]])
        before = np.concatenate([[0.0], sums[:-1]])
        keep = max(1, int((before < p * sums[-1]).sum()))
    chosen = np.zeros(x.size, dtype=bool)
    chosen[order[:keep]] = True
    if min_p is not None and min_p > 0:
        chosen &= w >= min(1.0, float(min_p))
    kept = np.where(chosen, w, 0.0)
    sums = np.cumsum(kept)
    z = sums[-1]
    goal = float(u) * z if u > 0 else 0.0
    over = np.flatnonzero(sums > goal)
    token = int(over[0]) if over.size else int(np.flatnonzero(kept > 0)[-1])
    margin = float(np.abs(sums - goal).min()) / z if goal > 0 else 1.0
    return token, float(y[token] - math.log(z)), margin


def _pages(tokens, page):
    return -(-tokens // page)


def append(lens, new, tables, free, count, page):
    tables = np.array(tables)
    columns = tables.shape[1]
    count = min(max(int(count), 0), len(free))
    granted, stopped = [], False
    for r, (a, b) in enumerate(zip(lens, new)):
        a, b = max(int(a), 0), max(int(b), 0)
        have, want = _pages(a, page), _pages(a + b, page)
        if want > columns or a + b > 2**31 - 1:
            granted.append(False)
            continue
        need = want - have
        stopped = stopped or need > count
        granted.append(need == 0 or not stopped)
        if need and not stopped:
            tables[r, have:want] = free[count - need:count][::-1]
            count -= need
    return tables, np.array(granted, dtype=bool), count


def slots(lens, new, tables, page, n):
    columns = tables.shape[1]
    slot = np.full(n, -1, dtype=np.int64)
    position, request = np.zeros(n, dtype=np.int32), np.full(n, -1, dtype=np.int32)
    offsets = np.concatenate([[0], np.cumsum(np.maximum(np.asarray(new, dtype=np.int64), 0))])
    for r in range(len(lens)):
        lo, hi = min(int(offsets[r]), n), min(int(offsets[r + 1]), n)
        at = max(int(lens[r]), 0) + np.arange(hi - lo, dtype=np.int64)
        col = at // page
        inside = col < columns
        held = np.full(hi - lo, -1, dtype=np.int64)
        if columns:
            held[inside] = tables[r, col[inside]]
        slot[lo:hi] = np.where(held >= 0, held * page + at % page, -1)
        position[lo:hi] = at
        request[lo:hi] = r
    return slot, position, request, offsets


def release(lens, finished, tables, free, count, page):
    free = np.array(free)
    columns = tables.shape[1]
    count = max(int(count), 0)
    for r in np.flatnonzero(finished):
        held = min(_pages(max(int(lens[r]), 0), page), columns)
        room = max(0, min(held, len(free) - count))
        free[count:count + room] = tables[r, :room]
        count += held
    return free, count
