"""Plain definitions of the calls around a serving step, for their tests (CPU): the step's tables with lists, the
sampling in float64.

Sampling: errors of a weight w_i before it is cut to a whole number of units (2^-46 of a power of two between the largest
weight and twice that): 1024 log2 of it is n + f with |f| <= 1/2, f from two fused products (2^-26 each) and the pair for
1024 log2 e / t (2^-49 of at most 2^22): less than 2^-24.6, which is 2^-35 of the weight; the power of f is off by 2^-33 (its
rounding) and 2^-35 + 2^-36 + 2^-37 (its sum and coefficients, the cubic term); the table by 2^-32; the product with it is cut
at 2^-31.  Together less than d = 2^-30.  Cut off: less than one unit, 2^-45 of the largest.  A border is a share x = c / S
of the kept mass: weights that are off by d each move it by at most 2 d x (1 - x) <= 2^-31, the cuts of n weights by n 2^-45
in c and in S.  border(n) = 2^-31 + n 2^-44 covers both.  `sample` raises where a border of its input lies nearer, so inputs
have to keep away from it (ties are exact on both sides).
probs: the ratio of a weight before the cut and the sum (2^-30 each, and the n 2^-45), rounded to fp32 once (2^-24; 2^-150 for
subnormal ones, half a step of 2^-149)."""
import math

import numpy as np

def border(n):
    return 2.0 ** -31 + n * 2.0 ** -44


class NearBorder(Exception):
    pass


def sample(z, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, u=0.0):
    """One row (float64 values of the logits): (token, probs)."""
    z = np.array(z, np.float64)
    z[np.isnan(z)] = -np.inf
    V = z.size
    probs = np.zeros(V)
    top = z.max()
    if not top > -np.inf:
        return -1, probs
    if not temperature > 0:
        t = int(np.argmax(z))
        probs[t] = 1.0
        return t, probs
    order = np.argsort(-z, kind="stable")
    order = order[z[order] > -np.inf]
    if 0 < top_k < V:
        order = order[:top_k]
    d = (z[order] - top)
    w = np.exp(d / temperature)
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        limit = top_p * w.sum()
        keep = before < limit
        keep[0] = True
        gap = np.abs(before[1:] - limit)
        # a border between equal weights that are exact on both sides is no matter of rounding
        exact = np.all(d == 0)
        if not exact and gap.size and gap.min() < border(V) * w.sum():
            raise NearBorder
        order, w = order[keep], w[keep]
    if min_p > 0:
        keep = w >= min(min_p, 1.0)
        near = np.abs(w / min(min_p, 1.0) - 1)
        if np.any((near < 2.0 ** -40) & (w != 1.0)):
            raise NearBorder
        order, w = order[keep], w[keep]
    by = np.argsort(order)
    order, w = order[by], w[by]
    c = np.cumsum(w)
    some = w > 2.0 ** -46
    hit = np.flatnonzero((c > u * c[-1]) & some)
    if 0 < u < 1 and np.abs(c[:-1] - u * c[-1]).min(initial=np.inf) < border(V) * c[-1] and not np.all(w == 1.0):
        raise NearBorder
    token = int(order[hit[0]]) if hit.size else int(order[np.flatnonzero(some)[-1]])
    probs[order] = w / c[-1]
    return token, probs


NO_PAGE, PAGE_RANGE, INDEX_RANGE = 0x40, 0x2, 0x4


def tables(cached, q, counts, keep, table, num_pages, stack, have, T):
    """The step's tables with lists; `table` (list of lists) and `stack` are updated.  Returns (seq_lens, counts, have,
    cu_q, positions, slots, error bits)."""
    max_pages, err = len(table[0]), 0
    have = max(0, min(num_pages, have))
    counts = [max(0, min(max_pages, c)) for c in counts]
    keep = [max(0, min(c, k)) for c, k in zip(counts, keep)]
    cached = [max(0, c) for c in cached]
    for b, n in enumerate(q):
        if n < 0:
            for i in range(keep[b], counts[b]):
                if have < num_pages:
                    stack[have] = table[b][i]
                    have += 1
                else:
                    err |= INDEX_RANGE
    cu, seq, mapped, pos, slots = [0], [], [], [], []

    def page(p):
        nonlocal err
        if 0 <= p < num_pages:
            return p
        err |= PAGE_RANGE
        return -1

    for b, n in enumerate(q):
        if n < 0:
            cu.append(cu[-1])
            seq.append(0)
            mapped.append(0)
            continue
        if n > T - cu[-1]:
            err |= INDEX_RANGE
            n = T - cu[-1]
        cu.append(cu[-1] + n)
        total = cached[b] + n
        seq.append(total)
        need = (total + 63) // 64
        if need > max_pages:
            err |= INDEX_RANGE
        got = counts[b]
        for i in range(counts[b], min(need, max_pages)):
            if have > 0:
                have -= 1
                table[b][i] = page(stack[have])
                got += 1
            else:
                err |= NO_PAGE
                table[b][i] = -1
        mapped.append(got)
        for p in range(cached[b], total):
            pos.append(p)
            i = p // 64
            slots.append(-1)
            if i < max_pages:
                if i < counts[b]:
                    g = page(table[b][i])
                else:
                    g = table[b][i]
                if g >= 0:
                    slots[-1] = g * 64 + p % 64
    pos += [0] * (T - len(pos))
    slots += [-1] * (T - len(slots))
    return seq, mapped, have, cu, pos, slots, err


def round_probs_bound(p):
    return (2.0 ** -24 + 2.0 ** -29 + p.size * 2.0 ** -45) * np.abs(p) + 2.0 ** -150
