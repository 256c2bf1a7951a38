"""Plain implementations for the serving operators' tests: the token draw in
64 bits, with the room that fp32 arithmetic has, and the block tables as loops
over rows."""
import math

import numpy as np

# Room of the fp32 arithmetic, from its roundings (u = 2^-24).
#   d = (x - M) / T : two or three roundings, |d| * 3u; exp's own error is below 4u, so
#     w's relative error is within (3 |d| + 4) u, taken as EPS * (|d| + 4) with EPS = 4u.
#   a sum of positive terms by at most 256 adds on any path: 256 u = 2^-16.
#   masses rounded to 2^-31: 2^-32 each.
EPS = 2.0 ** -22
SUM = 2.0 ** -16


def draw(x, noise, t=1.0, k=0, p=1.0, m=0.0):
    """One row.  Returns (tokens, logprob(token) -> (value, room)): the set of
    tokens that a correct fp32 draw may return -- almost always one -- and the
    log-probability of each with its room."""
    x = np.asarray(x, np.float64)
    alive = np.flatnonzero(~np.isnan(x) & (x > -np.inf))
    if alive.size == 0:
        return {-1}, lambda i: (-math.inf, 0.0)
    order = alive[np.lexsort((alive, -x[alive]))]
    top = x[order[0]]
    if noise is None or not t > 0:
        return {int(order[0])}, lambda i: (0.0, 0.0)
    v = x[order]
    with np.errstate(invalid="ignore", over="ignore"):
        d = np.where(v == top, 0.0, (v - top) / t)
    d = np.where(np.isnan(d), -np.inf, d)
    w = np.exp(d)
    near = EPS * (np.minimum(np.abs(d), 200.0) + 4)
    if 0 < k < order.size:
        order, d, w, near = order[:k], d[:k], w[:k], near[:k]
    sure = maybe = np.ones(order.size, bool)          # kept whatever the rounding; kept with luck
    if not p >= 1:
        ahead = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        total = w.sum()
        slack = (near * w).sum() + SUM * total + order.size * 2.0 ** -32
        bar = (p if p > 0 else 0.0) * total
        sure, maybe = ahead < bar - slack, ahead < bar + slack
    sure = sure & (w * (1 - near) >= m)
    maybe = maybe & (w * (1 + near) >= m)
    sure[0] = maybe[0] = True
    q = np.asarray(noise, np.float64)[order]
    score = np.where(maybe, w / q, -1.0)
    floor = np.max(np.where(sure, score * (1 - near - EPS), -1.0))
    good = maybe & (score * (1 + near + EPS) >= floor)
    tokens = {int(order[i]) for i in np.flatnonzero(good)}
    rest = w[1:][sure[1:]].sum()
    doubt = w[1:][maybe[1:] & ~sure[1:]].sum()
    room = (near[1:] * w[1:])[maybe[1:]].sum() + SUM * rest + doubt

    def logprob(i):
        at = int(np.flatnonzero(order == i)[0])
        value = d[at] - math.log1p(rest)
        return value, room / (1 + rest) + EPS * (abs(d[at]) + abs(value)) + 2.0 ** -140

    return tokens, logprob


def blocks(length, page):
    return -(-int(length) // page)


def extend(table, cached, fresh, pages, free, page):
    """In place on `table`; returns (granted, left)."""
    rows, width = table.shape
    granted = np.zeros(rows, np.uint8)
    free = min(max(int(free), 0), len(pages))
    at, short = free, False
    for r in range(rows):
        c, n = int(cached[r]), int(fresh[r])
        if c < 0 or n < 0 or blocks(c + n, page) > width:
            continue
        have, want = blocks(c, page), blocks(c + n, page)
        if want == have:
            granted[r] = 1
            continue
        if short or want - have > at:
            short = True
            continue
        for j in range(have, want):
            at -= 1
            table[r, j] = pages[at]
        granted[r] = 1
    return granted, at


def slots(table, cached, fresh, page, tokens, granted=None):
    rows, width = table.shape
    starts = np.zeros(rows + 1, np.int64)
    out = np.full(tokens, -1, np.int64)
    positions, ids = np.full(tokens, -1, np.int64), np.full(tokens, -1, np.int64)
    g = 0
    for r in range(rows):
        n = max(0, int(fresh[r])) if granted is None or granted[r] else 0
        for i in range(min(n, max(0, tokens - g))):
            pos = int(cached[r]) + i
            ids[g + i] = r
            if 0 <= pos <= 2**31 - 1:
                positions[g + i] = pos
                b = pos // page
                if b < width and table[r, b] >= 0:
                    out[g + i] = int(table[r, b]) * page + pos % page
        g += n
        starts[r + 1] = min(g, 2**31 - 1)
    return starts, out, positions, ids


def release(table, cached, done, pages, free, page):
    """In place on `pages`; returns the stack's height."""
    rows, width = table.shape
    free = min(max(int(free), 0), len(pages))
    for r in range(rows):
        if not done[r] or cached[r] <= 0:
            continue
        n = min(blocks(cached[r], page), width)
        if free + n > len(pages):
            break
        pages[free:free + n] = table[r, :n]
        free += n
    return free
