"""Plain 64-bit statements of the paged-cache operators, for the tests (host only)."""

import math

import numpy as np
import torch

# Rounding of a value to the type (half an ulp, relative).
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def plan(ctx, new, page, table, free, head, capacity):
    """(table, row_start, slots, positions, request, info) from plain lists."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    flags, taken, start, slots, positions, request = 0, 0, [0], [], [], []
    for b, (c, n) in enumerate(zip(ctx, new)):
        if c < 0 or n < 0:
            flags |= 8
        c, n = max(c, 0), max(n, 0)
        if -(-(c + n) // page) > width:
            flags |= 2
        for at in range(min(-(-c // page), width), min(-(-(c + n) // page), width)):
            if head + taken < len(free):
                table[b][at] = free[head + taken]
            else:
                table[b][at] = -1
                flags |= 1
            taken += 1
        for i in range(n):
            p = c + i
            pg = table[b][p // page] if p // page < width else -1
            slots.append(pg * page + p % page if pg >= 0 else -1)
            positions.append(p)
            request.append(b)
        start.append(start[-1] + n)
    total = len(slots)
    if total > capacity:
        flags |= 4
    pad = max(0, capacity - total)
    taken = min(taken, len(free) - head)
    return (table, start, (slots + [-1] * pad)[:capacity], (positions + [0] * pad)[:capacity],
            (request + [-1] * pad)[:capacity], [total, taken, head + taken, flags])


def attention(q, k, v, table, page, ctx, new, seen, scale):
    """(out, lse, weight) in 64 bits: q [T, Hq, D], k and v [pages, page, H, D] (float64
    arrays), seen(b, i, j): whether new token i of request b sees new token j.  ``weight`` is
    sum p |v| / sum p, what a relative error of the probabilities is multiplied by."""
    t, hq, d = q.shape
    h = k.shape[2]
    group = hq // h
    out, lse, weight = np.zeros(q.shape), np.full((t, hq), -np.inf), np.zeros(q.shape)
    row = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        pos = np.arange(c + n)
        pages = np.asarray(table[b], dtype=np.int64)[pos // page] if c + n else pos
        kb, vb = k[pages, pos % page], v[pages, pos % page]          # [L, H, D]
        for i in range(n):
            keep = np.array([True] * c + [bool(seen(b, i, j)) for j in range(n)])
            if keep.any():
                for x in range(hq):
                    kk, vv = kb[keep, x // group], vb[keep, x // group]
                    with np.errstate(all="ignore"):
                        s = kk @ q[row, x] * scale
                        m = s.max()
                        if m == -np.inf:
                            continue
                        p = np.exp(s - m)
                        lse[row, x] = m + math.log(p.sum()) if np.isfinite(p.sum()) else p.sum()
                        out[row, x] = p @ vv / p.sum()
                        weight[row, x] = p @ np.abs(vv) / p.sum()
            row += 1
    return out, lse, weight


def attention_bounds(q, k, dim, keys, scale, dtype, ref, weight, lse):
    """What the kernel's roundings can add up to, element by element: (of out, of lse).

    A score is a sum of ``dim`` products in 32 bits, so it is off by at most (dim + 2) 2^-24
    times the sum of its products' absolute values (bounded here by the largest norms), plus
    its scaling and the exponential's argument (2 roundings of |s|, itself within that bound).
    A probability is then off by that and the exponential's 2^-21, relatively; the sums over
    the keys add ``keys`` 2^-24 each; the probability is rounded to the cache's type once for
    the second product, and the output once."""
    unit, eps = UNIT[dtype], 2.0 ** -24
    largest = abs(scale) * np.sqrt((q ** 2).sum(-1)).max() * np.sqrt((k ** 2).sum(-1)).max()
    score = (dim + 6) * eps * largest
    rel = score + 2.0 ** -21 + (keys + 8) * eps
    of_out = weight * (unit + 2 * rel) * (1 + unit) + unit * np.abs(ref) + 2.0 ** -24
    of_lse = rel + 4 * eps * np.abs(np.where(np.isfinite(lse), lse, 0)) + 2.0 ** -20
    return of_out, of_lse
