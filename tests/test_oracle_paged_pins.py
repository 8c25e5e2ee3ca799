"""The paged oracle against other things than itself: the dense oracle, hand-made
tables and the invariants of the page counts.  CPU only."""

import random

import numpy as np
import pytest
import torch

import oracle
from oracle import paged


def _dense_to_pages(x, ps, order):
    """[T, Hkv, D] into pages in the given order; unused slots NaN."""
    pages = torch.full((len(order), ps) + tuple(x.shape[1:]), float("nan"), dtype=x.dtype)
    row = [-1] * len(order)
    for j in range(-(-x.shape[0] // ps)):
        part = x[j * ps:(j + 1) * ps]
        row[j] = order[j]
        pages[order[j], :part.shape[0]] = part
    return pages, row


@pytest.mark.parametrize("window", [0, 1, 5, 129])
@pytest.mark.parametrize("n", [1, 7, 40])
def test_chunk_equals_the_last_rows_of_a_dense_prefill(window, n):
    g = torch.Generator().manual_seed(n + window)
    T, hq, hkv, ps = 40, 4, 2, 16
    q = torch.randn((T, hq, 192), generator=g, dtype=torch.float64)
    k = torch.randn((T, hkv, 192), generator=g, dtype=torch.float64)
    v = torch.randn((T, hkv, 128), generator=g, dtype=torch.float64)
    sinks = torch.randn(hq, generator=g, dtype=torch.float64)
    want, want_lse = oracle.prefill(q, k, v, sinks, window, [0, T])
    kp, row = _dense_to_pages(k, ps, [5, 0, 3, 1, 2, 4])
    vp, _ = _dense_to_pages(v, ps, [5, 0, 3, 1, 2, 4])
    if window:  # pages behind the window may be gone
        for j in range(max(0, T - n - window + 1) // ps):
            row[j] = -1
    out, lse, mass = paged.paged_attention(q[T - n:], kp, vp, [row], [0, n], [T], window, sinks)
    assert np.allclose(out, want[T - n:], atol=1e-12)
    assert np.allclose(lse, want_lse[:, T - n:], atol=1e-12)
    assert np.all(mass + 1e-12 >= np.abs(out))


def test_append_writes_the_slots_of_its_positions_only():
    g = torch.Generator().manual_seed(0)
    q = torch.randn((3, 2, 192), generator=g)
    k = torch.randn((3, 1, 192), generator=g)
    v = torch.randn((3, 1, 128), generator=g)
    kp, vp = torch.zeros((4, 16, 1, 192)), torch.zeros((4, 16, 1, 128))
    qo, ko, vo = paged.paged_append(q, k, v, kp, vp, [[2, 0], [3, -1]], [0, 2, 3], [17, 1], 10000.0)
    written = {(p, s) for p in range(4) for s in range(16) if vo[p, s].any()}
    assert written == {(2, 15), (0, 0), (3, 0)}
    assert np.allclose(qo[2], q[2].numpy()) and np.allclose(ko[3, 0], k[2].numpy())  # position 0 turns nothing
    assert np.allclose(np.linalg.norm(qo, axis=-1), np.linalg.norm(q.numpy(), axis=-1), rtol=1e-6)


def _holders(table, pool):
    refs = [0] * pool
    for row in table:
        for e in row:
            if e >= 0:
                refs[e] += 1
    return refs


@pytest.mark.parametrize("seed", range(20))
def test_a_run_of_bookkeeping_keeps_counts_and_contents(seed):
    """Random holds, forks and compactions: the counts stay the table's, and what each
    sequence wrote at each position stays there."""
    r = random.Random(seed)
    ps, pool, B, M = 4, 24, 4, 6
    refs, table, lens = [0] * pool, [[-1] * M for _ in range(B)], [0] * B
    data, said = [[None] * ps for _ in range(pool)], [[] for _ in range(B)]
    for step in range(60):
        what = r.choice(["grow", "grow", "cut", "fork", "compact"])
        if what == "grow":
            new = [min(M * ps, n + r.randint(0, 3)) for n in lens]
            refs2, table2, moves, info = paged.page_hold(refs, table, new, ps, write_from=lens)
            if info[0]:
                assert (refs2, table2) == (refs, table)
                continue
            refs, table = refs2, table2
            for s, d in moves:
                if s >= 0:
                    data[d] = list(data[s])
            for b in range(B):
                for p in range(lens[b], new[b]):
                    said[b].append((step, b, p))
                    data[table[b][p // ps]][p % ps] = said[b][-1]
            lens = new
        elif what == "cut":
            lens = [r.randint(max(0, n - 3), n) for n in lens]
            said = [s[:n] for s, n in zip(said, lens)]
            refs, table, moves, info = paged.page_hold(refs, table, lens, ps)
            assert info[0] == 0 and moves == [[-1, -1]] * B
        elif what == "fork":
            parent = [r.choice([b, b, r.randrange(-1, B)]) for b in range(B)]
            refs, table = paged.page_fork(refs, table, parent)
            lens = [lens[p] if p >= 0 else 0 for p in parent]
            said = [list(said[p]) if p >= 0 else [] for p in parent]
        else:
            refs, table, moves, info = paged.page_compact(refs, table, r.randint(0, 5))
            for s, d in moves:
                if s >= 0:
                    data[d] = list(data[s])
        assert refs == _holders(table, pool)
        for b in range(B):
            assert [data[table[b][p // ps]][p % ps] for p in range(lens[b])] == said[b]


def test_hold_with_a_window_releases_what_lies_behind_it():
    refs, table, moves, info = paged.page_hold([0] * 8, [[-1] * 6], [20], 4)
    assert table == [[0, 1, 2, 3, 4, -1]] and refs == [1, 1, 1, 1, 1, 0, 0, 0] and info == [0, 3]
    refs, table, moves, info = paged.page_hold(refs, table, [24], 4, first=[10])
    assert table == [[-1, -1, 2, 3, 4, 0]] and info == [0, 4]


def test_hold_without_enough_pages_changes_nothing():
    refs, table = [1, 1, 0], [[0, -1, -1], [1, -1, -1]]
    got = paged.page_hold(refs, table, [12, 0], 4, first=[0, 0])
    assert got == ([1, 1, 1], [[0, 1, 2], [-1, -1, -1]], [[-1, -1], [-1, -1]], [0, 0])
    got = paged.page_hold(refs, table, [12, 4], 4)
    assert got == (refs, table, [[-1, -1], [-1, -1]], [1, 1])


def test_compact_moves_the_end_to_the_holes():
    refs, table, moves, info = paged.page_compact([0, 2, 0, 1, 0, 1], [[1, 5], [1, 3]], 5)
    assert info == [2, 3] and moves[:2] == [[3, 0], [5, 2]]
    assert refs == [1, 2, 1, 0, 0, 0] and table == [[1, 2], [1, 0]]
