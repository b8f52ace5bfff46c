"""CPU oracle of the key/value cache operators, in 64 bits.

TEST INFRASTRUCTURE ONLY, as the rest of this package: only ``tests/`` imports it,
and the CUDA library shares no code with it.

* ``plan``: pages and slots, request after request, with the free pages as a queue.
* ``append``: e4m3 codes with one power-of-two scale per page and head.
* ``attend``: softmax(scale q k^T) v over one row's visible keys, with the bounds on
  the rounding errors of a 32-bit computation that the tests compare against.
"""
from __future__ import annotations

import numpy as np

SHORT_OF_PAGES, BAD_LENGTH, SHORT_OF_ROWS, BAD_PATH, BAD_INDEX = 1, 2, 4, 8, 16


def _blocks(x, page):
    return -(-int(x) // page)


def plan(old, delta, extra, table, ring, head, count, page, max_rows, path=None, path_rows=0):
    """dict of len, table, ring, head, count, row_start, slot, pos, src, status."""
    n, width, n_pages = len(old), table.shape[1], len(ring)
    delta = [0] * n if delta is None else [int(d) for d in delta]
    new = [max(0, int(o) + d + extra) for o, d in zip(old, delta)]
    status, rows, take, give = 0, 0, 0, 0
    for q in range(n):
        if old[q] < 0 or _blocks(old[q], page) > width or _blocks(new[q], page) > width:
            status |= BAD_LENGTH
            continue
        r = max(0, new[q] - int(old[q]))
        rows += r
        take += max(0, _blocks(new[q], page) - _blocks(old[q], page))
        give += max(0, _blocks(old[q], page) - _blocks(new[q], page))
        if path is not None and r:
            if r - 1 > path.shape[1] or any(not 0 <= s < path_rows for s in path[q, :r - 1]):
                status |= BAD_PATH
    if take > count:
        status |= SHORT_OF_PAGES
    if give > n_pages - count:
        status |= BAD_INDEX
    if rows > max_rows:
        status |= SHORT_OF_ROWS
    table, ring = table.copy(), ring.copy()
    slot, pos, src = (np.full(max_rows, -1, np.int64) for _ in range(3))
    start = [0]
    if status:
        return dict(len=list(map(int, old)), table=table, ring=ring, head=head, count=count,
                    row_start=[0] * (n + 1), slot=slot, pos=pos, src=src, status=status)
    put, took = head + count, 0
    for q in range(n):
        for b in range(_blocks(old[q], page), _blocks(new[q], page)):
            table[q, b] = ring[(head + took) % n_pages]
            took += 1
        for b in range(_blocks(new[q], page), _blocks(old[q], page)):
            ring[put % n_pages] = table[q, b]
            put += 1
        t = start[-1]
        for j, p in enumerate(range(int(old[q]), new[q])):
            pos[t], slot[t] = p, int(table[q, p // page]) * page + p % page
            src[t] = t if path is None else q * path_rows + (path[q, j - 1] if j else 0)
            t += 1
        start.append(t)
    return dict(len=new, table=table, ring=ring, head=(head + take) % n_pages, count=count - take + give,
                row_start=start, slot=slot, pos=pos, src=src, status=0)


def round_e4m3(x):
    """Nearest e4m3 value (ties to even) of finite |x| <= 448; NaN stays NaN."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(np.where(np.isnan(x), 1.0, x))
    unit = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(x / unit) * unit


def pow2_scale(amax):
    """Smallest power of two s in [2^-126, 2^120] with 448 s >= amax."""
    if amax == 0:
        return 2.0 ** -126
    m, e = np.frexp(float(amax) / 448.0)
    return float(np.ldexp(1.0, int(min(max(e - (1 if m == 0.5 else 0), -126), 120))))


def append(codes, scale, x, slots, src, page):
    """codes [n_pages, n_kv, page, hd] (values, float64), scale [n_pages, n_kv], both changed in place.
    x [rows, n_kv, hd]; slots per row (negative: skipped); src: row of x per row, or None."""
    t = 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        run = [t]
        while t + len(run) < len(slots) and slots[t + len(run)] == slots[t] + len(run) and slots[t + len(run)] % page:
            run.append(t + len(run))
        pg, off = slots[t] // page, slots[t] % page
        rows = np.array([r if src is None else src[r] for r in run])
        for h in range(codes.shape[1]):
            y = x[rows, h].astype(np.float64)
            fin = np.isfinite(y)
            now = pow2_scale(np.abs(np.where(fin, y, 0)).max())
            if off:
                now = max(now, float(scale[pg, h]))
                codes[pg, h, :off] = round_e4m3(codes[pg, h, :off] * (float(scale[pg, h]) / now))
            codes[pg, h, off:off + len(run)] = round_e4m3(np.where(fin, y, np.nan) / now)
            scale[pg, h] = now
        t += len(run)


def attend(q, k, v, see, scale, weight_unit):
    """One head's rows q [R, hd] over keys k, v [T, hd] with see [R, T] -> out [R, hd], lse [R], and
    their tolerances.

    A product of hd terms in 32 bits is off by at most hd 2^-24 B, B = scale sum |q||k|; so are z and
    lse (and a sum of T terms e^z adds up to T 2^-24 at worst, 2^-14 here).  The weights are then off by
    that and by their own rounding to a 16-bit type: weight_unit, half its spacing at 1, is 2^-8 for the 8
    significant bits of bf16 and 2^-11 for the 11 of fp16.  The output is off by its rounding to bf16, 2^-8 |out|.
    (The bound holds for any signs; the weights' errors hardly ever add up so.)"""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    R, hd = q.shape
    out, lse = np.zeros((R, hd)), np.full(R, -np.inf)
    tol_out, tol_lse = np.zeros((R, hd)), np.zeros(R)
    for r in range(R):
        s = np.asarray(see[r], bool)
        if not s.any():
            continue
        z = scale * (k[s] @ q[r])
        top = z.max()
        p = np.exp(z - top)
        out[r], lse[r] = p @ v[s] / p.sum(), top + np.log(p.sum())
        off = hd * 2.0 ** -24 * np.abs(scale) * (np.abs(k[s]) @ np.abs(q[r])).max() + 2.0 ** -14
        weight = p @ np.abs(v[s]) / p.sum()
        tol_lse[r] = off
        tol_out[r] = 2.0 ** -8 * np.abs(out[r]) + (weight_unit + 2 * off) * 1.02 * weight + 1e-30
    return out, lse, tol_out, tol_lse
