"""Paged cache, fp64 / integer oracle: attention of a chunk over pages, the
chunk's rotation and write, and the page bookkeeping.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Written from the definitions, one row and one table entry at a time; shares no
code with the GPU path.  A sequence of length L (its n new tokens included)
keeps position p in slot ``p % page_size`` of page ``table[b][p // page_size]``;
query i of the chunk sits at position L - n + i.
"""

from __future__ import annotations

import math

import numpy as np

from .attention import _f64
from .rope import rope


def gather(pages, row, lo, hi):
    """Positions [lo, hi) of one sequence as a dense [hi - lo, Hkv, D] float64 array;
    a position without a page reads as zeros."""
    ps = pages.shape[1]
    out = np.zeros((hi - lo,) + tuple(pages.shape[2:]))
    for j in range(lo // ps, -(-hi // ps) if hi > lo else lo // ps):
        a, b = max(lo, j * ps), min(hi, (j + 1) * ps)
        if 0 <= row[j] < pages.shape[0]:
            out[a - lo:b - lo] = _f64(pages[int(row[j]), a - j * ps:b - j * ps])
    return out


def paged_attention(q, k_pages, v_pages, table, cu, lens, window, sinks, scale=None, v_scale=1.0):
    """Returns (out [Nt,Hq,Dv], lse [Hq,Nt], mass [Nt,Hq,Dv]) in float64, mass being
    v_scale * sum_j w_j |v_j| (what a relative rounding of the weights can move).
    Rows that belong to no sequence are NaN."""
    q = _f64(q)
    nt, hq, dqk = q.shape
    hkv, dv = k_pages.shape[2], v_pages.shape[3]
    g = hq // hkv
    scale = 1.0 / math.sqrt(dqk) if scale is None else scale
    out = np.full((nt, hq, dv), np.nan)
    mass = np.full((nt, hq, dv), np.nan)
    lse = np.full((hq, nt), np.nan)
    for b, L in enumerate(int(x) for x in lens):
        n = int(cu[b + 1]) - int(cu[b])
        if n == 0:
            continue
        lo0 = max(0, L - n - window + 1) if window else 0
        k, v = gather(k_pages, table[b], lo0, L), gather(v_pages, table[b], lo0, L)
        for i in range(n):
            p, t = L - n + i, int(cu[b]) + i
            lo = max(0, p - window + 1) if window else 0
            kk, vv = k[lo - lo0:p + 1 - lo0], v[lo - lo0:p + 1 - lo0]
            for h in range(hq):
                s = scale * (kk[:, h // g] @ q[t, h])
                sig = -math.inf if sinks is None else float(sinks[h])
                m = max(sig, s.max())
                e = np.exp(s - m)
                z = e.sum() + math.exp(sig - m)
                w = e / z
                out[t, h] = v_scale * (w @ vv[:, h // g])
                mass[t, h] = abs(v_scale) * (w @ np.abs(vv[:, h // g]))
                lse[h, t] = m + math.log(z)
    return out, lse, mass


def paged_append(q, k_new, v_new, k_pages, v_pages, table, cu, lens, theta, rotary_dim=None):
    """Returns (q, k_pages, v_pages) in float64 after the call."""
    q, k, v = _f64(q).copy(), _f64(k_new), _f64(v_new)
    kp, vp = _f64(k_pages).copy(), _f64(v_pages).copy()
    ps = kp.shape[1]
    for b, L in enumerate(int(x) for x in lens):
        lo, hi = int(cu[b]), int(cu[b + 1])
        pos = np.arange(L - (hi - lo), L)
        q[lo:hi] = rope(q[lo:hi], pos, theta, rotary_dim)
        kr = rope(k[lo:hi], pos, theta, rotary_dim)
        for i, p in enumerate(pos):
            page = int(table[b][p // ps])
            if 0 <= page < kp.shape[0]:
                kp[page, p % ps] = kr[i]
                vp[page, p % ps] = v[lo + i]
    return q, kp, vp


def page_hold(refs, table, lens, page_size, first=None, write_from=None):
    """Returns (refs, table, moves, info) as lists; the inputs are left alone."""
    refs0, table0 = [int(x) for x in refs], [[int(x) for x in r] for r in table]
    refs, table = list(refs0), [list(r) for r in table0]
    bounds = []
    for b, row in enumerate(table):
        f = 0 if first is None else int(first[b])
        w = int(lens[b]) if write_from is None else int(write_from[b])
        if int(lens[b]) < 0 or f < 0 or w < 0 or int(lens[b]) > len(row) * page_size:
            bounds.append(None)  # left as it is
            continue
        bounds.append((f // page_size, -(-int(lens[b]) // page_size), w))
    for row, bd in zip(table, bounds):
        for j in range(len(row)):
            if bd and not bd[0] <= j < bd[1]:
                if row[j] >= 0:
                    refs[row[j]] -= 1
                row[j] = -1
    need = []
    for b, (row, bd) in enumerate(zip(table, bounds)):
        for j in range(len(row)):
            if not bd or not bd[0] <= j < bd[1]:
                continue
            if row[j] < 0:
                need.append((b, j))
            elif write_from is not None and j >= bd[2] // page_size and refs[row[j]] > 1:
                need.append((b, j))
    free = [p for p, c in enumerate(refs) if c == 0]
    moves = [[-1, -1] for _ in table]
    if len(need) > len(free):
        return refs0, table0, moves, [len(need) - len(free), refs0.count(0)]
    for (b, j), page in zip(need, free):
        old = table[b][j]
        if old >= 0:
            refs[old] -= 1
            if j * page_size < bounds[b][2]:
                moves[b] = [old, page]
        table[b][j] = page
        refs[page] = 1
    return refs, table, moves, [0, refs.count(0)]


def page_fork(refs, table, parent):
    refs = [int(x) for x in refs]
    m = len(table[0]) if len(table) else 0
    out = [[int(x) for x in table[p]] if 0 <= p < len(table) else [-1] * m for p in (int(x) for x in parent)]
    for rows, d in ((table, -1), (out, 1)):
        for row in rows:
            for e in row:
                if e >= 0:
                    refs[int(e)] += d
    return refs, out


def page_compact(refs, table, max_moves):
    refs = [int(x) for x in refs]
    u = sum(c > 0 for c in refs)
    src = [p for p, c in enumerate(refs) if c > 0 and p >= u]
    dst = [p for p, c in enumerate(refs) if c <= 0 and p < u]
    pairs = list(zip(src, dst))[:max_moves]
    to = dict(pairs)
    for s, d in pairs:
        refs[d], refs[s] = refs[s], 0
    out = [[to.get(int(e), int(e)) for e in row] for row in table]
    return refs, out, [list(p) for p in pairs] + [[-1, -1]] * (max_moves - len(pairs)), [len(pairs), u]
