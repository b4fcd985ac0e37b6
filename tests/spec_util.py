"""Plain forms of a speculative step's operators on the host: the plan in Python's whole numbers, the verification in
exact ones, the probabilities in 64 bits."""
from fractions import Fraction

import numpy as np


def plan(P, row0, kv_len, table, held, pinned, take, grow, ring, state, rows, max_tokens):
    """One sequence after the other.  Returns (row0, kv_len, held, granted, state, positions, slots, seq_of); table and
    ring change in place.  Sequences whose numbers make no sense keep their tokens and get nothing."""
    head, free = state
    cap, width = len(ring), table.shape[1]
    queue = [ring[(head + i) % cap] for i in range(free)]
    back, full, used = [], False, 0
    out = ([0], [], [], [], [], [], [])
    for b in range(len(kv_len)):
        n = row0[b + 1] - row0[b]
        kept, count, pages = kv_len[b], 0, held[b]
        sane = row0[b] >= 0 and 0 <= n <= kv_len[b] and 0 <= held[b] <= width and pinned[b] >= 0
        if sane and take[b] < 0:
            back += table[b, pinned[b]:held[b]].tolist()
            kept, pages = 0, 0
        elif sane and take[b] <= n and 0 <= grow[b] <= max_tokens and -(-(kv_len[b] - n + take[b] + grow[b]) // P) <= width:
            kept, count = kv_len[b] - n + take[b], grow[b]
            need = max(0, -(-(kept + count) // P) - pages) if count else 0
            full = full or used + need > free or out[0][-1] + count > rows
            if full:
                count = need = 0
            for _ in range(need):
                table[b, pages] = queue[used]
                pages, used = pages + 1, used + 1
        else:
            kept = max(kept, 0)
            full = full or used > free
        for t in range(kept, kept + count):
            out[4].append(t)
            out[5].append(table[b, t // P] * P + t % P)
            out[6].append(b)
        for o, v in zip(out, (out[0][-1] + count, kept + count, pages, count)):
            o.append(v)
    for i, x in enumerate(back):
        ring[(head + free + i) % cap] = x
    return (*out[:4], [(head + used) % cap, free - used + len(back)], *out[4:])


def units(x):
    """Weights in units of 2^-44, halves to even, of values inside [0, 1] (a NaN: 0)."""
    x = np.nan_to_num(x.astype(np.float64), nan=0.0, posinf=1.0, neginf=0.0).clip(0.0, 1.0)
    return np.rint(x * 2.0 ** 44).astype(np.int64)


def unit_interval(x):
    return min(max(float(x), 0.0), 1.0) if x == x else 0.0


def verify(p, q, tokens, row0, accept, sample):
    """(next, take) with exact sums; None in `next` where it is left as it was."""
    V = p.shape[1]
    nxt, take = [None] * p.shape[0], []
    for a, b in zip(row0, row0[1:]):
        if a == b:
            take.append(0)
            continue
        r, d = a, -1
        while r + 1 < b:
            d = int(tokens[r + 1])
            if not 0 <= d < V:
                break
            pd, qd = unit_interval(p[r, d]), 1.0 if q is None else unit_interval(q[r, d])
            if not Fraction(unit_interval(accept[r])) * Fraction(qd) < Fraction(pd):
                break
            nxt[r] = d
            r += 1
        w = target = units(p[r])
        if r + 1 < b:
            if q is not None:
                w = np.maximum(target - units(q[r]), 0)
            else:
                w = target.copy()
                if 0 <= d < V:
                    w[d] = 0
        if w.sum() == 0:
            w = target
        cum = np.cumsum(w)
        total = int(cum[-1])
        at = min(int(Fraction(unit_interval(sample[r])) * total), total - 1)
        nxt[r] = int(np.searchsorted(cum, at, side="right")) if total > 0 else -1
        for i in range(r + 1, b):
            nxt[i] = -1
        take.append(r - a + 1)
    return nxt, take


def probs(x, inv):
    """(probabilities, bound of |gpu - p|) of logits x [rows, V], in 64 bits.

    The bound follows the arithmetic, with u = 2^-24 and t = (x - ref) inv <= 0 of a value (ref: its warp's maximum) or of a
    warp's maximum (ref: the row's): the difference, log2 e, its product with inv and the product of the two are four
    roundings at most, 4 u |t| of the exponential, which is off by 2^-22 (the instruction's) and u for its last step.  A
    value's t and its warp's add up to the value's in the row.  Sums of positive terms: 32 of a thread at most in one chain
    (16 in each of two where no value is NaN), 2 to join its four, 5 of a warp, 4 products added by a lane over the warps'
    sums, 5 of the lanes; the quotient, the factor and the product 3 more: 51, under the 99 that are taken.  What is below
    2^-126 of a warp's maximum may be 0."""
    u = 2.0 ** -24
    x = x.astype(np.float64)
    out, bound = np.zeros_like(x), np.full_like(x, 2.0 ** -125)
    for r in range(x.shape[0]):
        v = np.where(np.isnan(x[r]), -np.inf, x[r])
        top, k = v.max(), 0.0 if not inv[r] >= 0 else float(inv[r])
        if top == -np.inf:
            continue
        if k == np.inf:
            out[r, int(np.argmax(v == top))] = 1.0
            continue
        if top == np.inf:
            t = np.where(v == np.inf, 0.0, -np.inf)
        else:
            t = np.where(v == -np.inf, -np.inf, (np.where(v == -np.inf, 0.0, v) - top) * k)
        e = np.exp(t)
        p = e / e.sum()
        size = np.where(np.isinf(t), 0.0, np.abs(t))
        rel = lambda s: 4 * u * s + 2 * (2.0 ** -22 + u)   # noqa: E731
        mean = (p * rel(size)).sum()
        out[r], bound[r] = p, bound[r] + 1.01 * p * (rel(size) + mean + 99 * u)
    return out, bound
