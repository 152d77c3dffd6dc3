"""Oracle of a serving step's calls: slots (plain integers, sequence by
sequence), adapters (fp64) and sampling (fp64, sorted).  Written from the
definitions in include/wq.h; shares no code with the HIP path."""

import math

import numpy as np


def kv_slots(page, pages, table, lens, new, free, used, tokens):
    """-> (slots, positions, seq_of, lens_out, last, used_out, table) as int32 arrays."""
    table = np.array(table, dtype=np.int32)
    slots, positions, seq_of = (np.full(tokens, -1, np.int32) for _ in range(3))
    lens_out, last = np.array(lens, dtype=np.int32), np.full(len(lens), -1, np.int32)
    room = len(free) - used if 0 <= used <= len(free) else 0
    row, asked, taken = 0, 0, 0
    for s, (held, add) in enumerate(zip(lens, new)):
        held, add = max(int(held), 0), max(int(add), 0)
        first, row = row, row + add
        if row > tokens or held + add > min(table.shape[1] * page, 2 ** 31 // page * page - page):
            continue
        old = -(-held // page)
        need = -(-(held + add) // page) - old
        place, asked = asked, asked + need
        if need and asked > room:
            continue
        for j in range(need):
            table[s, old + j] = free[used + place + j]
        taken = max(taken, asked if need else 0)
        lens_out[s] = held + add
        if add:
            last[s] = row - 1
        for i in range(add):
            p = held + i
            number = int(table[s, p // page])
            slots[first + i] = number * page + p % page if 0 <= number < pages else -1
            positions[first + i], seq_of[first + i] = p, s
    return slots, positions, seq_of, lens_out, last, np.array([used + taken], np.int32), table


def lora(a, b, x, ids, base, scales=None):
    """One linear: y in fp64, and the bound of what 32-bit sums, two fp16 parts
    of A x and no rounding of y may be off, element by element."""
    y = np.array(base, dtype=np.float64)
    off = np.zeros_like(y)
    eps = 2.0 ** -24
    for r, d in enumerate(ids):
        if not 0 <= d < len(a):
            continue
        f = 1.0 if scales is None else float(scales[d])
        aa, bb, xx = a[d].astype(np.float64), b[d].astype(np.float64), x[r].astype(np.float64)
        t = aa @ xx
        # k products, exact in 32 bits, and their sum in any order; the scale's rounding; the two parts
        dt = (len(xx) + 2) * eps * (np.abs(aa) @ np.abs(xx)) + 2.0 ** -21 * np.abs(t).max()
        y[r] += f * (bb @ t)
        both = np.abs(bb) @ np.abs(t)
        off[r] = abs(f) * (np.abs(bb) @ dt + (len(t) * 2 + 4) * eps * both) + 2 * eps * np.abs(y[r])
    return y, off


def kept(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row's tokens that can be drawn, by index, and their weights (the largest 1); temperature above 0."""
    x = np.asarray(logits, dtype=np.float64)
    place = np.flatnonzero(x > -math.inf)          # neither NaN nor -infinity
    place = place[np.lexsort((place, -x[place]))]
    if not len(place):
        return place, np.zeros(0)
    top = x[place[0]]
    with np.errstate(over="ignore", invalid="ignore"):
        w = np.where(x[place] == top, 1.0, np.exp((x[place] - top) / float(temperature)))
    w[np.isnan(w)] = 0.0
    if 0 < top_k < len(place):
        place, w = place[:top_k], w[:top_k]
    if top_p < 1:
        before = np.concatenate(([0.0], np.cumsum(w)[:-1]))
        keep = before < max(float(top_p), 0.0) * w.sum()
        keep[0] = True
        place, w = place[keep], w[keep]
    if min_p > 0:
        keep = w >= min(float(min_p), 1.0)
        place, w = place[keep], w[keep]
    order = np.argsort(place)
    return place[order], w[order]


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row -> (id, logprob)."""
    x = np.asarray(logits, dtype=np.float64)
    if not (x > -math.inf).any():
        return -1, -math.inf
    if not temperature > 0:
        return int(np.argmax(np.where(np.isnan(x), -math.inf, x))), 0.0
    place, w = kept(logits, temperature, top_k, top_p, min_p)
    up_to = np.cumsum(w)
    u = min(max(float(u), 0.0), 1.0) if u == u else 0.0
    i = min(int(np.searchsorted(up_to, u * up_to[-1], side="right")), int(np.flatnonzero(w)[-1]))
    return int(place[i]), math.log(w[i] / up_to[-1])
