"""The plain pool model itself, on the CPU: its invariants, by hand-worked
cases, so that the GPU calls are held to something that has been checked."""
import numpy as np
import pytest

from _pool import POOL, REFS, ROW, Pool


def counts(p):
    """References as the tables hold them."""
    n = np.zeros(p.N, np.int64)
    for r in range(p.rows):
        for e in p.table[r, :p.blocks(p.lens[r])]:
            if e >= 0:
                n[e] += 1
    return n


def test_fork_shares_whole_pages_and_copies_the_last():
    p = Pool(8, 3, 4, 4, [16])
    p.fill_row(0, 6, [5, 2])
    p.fork([0, 0], [2, 1])
    assert p.table[2, :2].tolist() == [5, 0] and p.table[1, :2].tolist() == [5, 1]
    assert p.refs.tolist() == [1, 1, 1, 0, 0, 3, 0, 0]
    assert (p.caches[0][0] == p.caches[0][2]).all() and (p.caches[0][1] == p.caches[0][2]).all()
    assert p.lens.tolist() == [6, 6, 6] and p.err == 0
    p.free([2, 1, 2])
    assert p.refs.tolist() == [0, 0, 1, 0, 0, 1, 0, 0] and p.err == 0


def test_fork_refusals():
    p = Pool(3, 4, 4, 4, [16])
    p.fill_row(0, 6, [0, 1])
    p.fork([0, 0, 0, 9, 0], [1, 1, 0, 2, 3])  # ok, named twice, in use, out of range, no page
    assert p.err == ROW | POOL and p.lens.tolist() == [6, 6, 0, 0]


def test_window_free_keeps_what_can_be_seen():
    p = Pool(16, 1, 10, 4, [4])
    p.fill_row(0, 38)
    p.free([0], window=9, sinks=5)  # tokens 0..4 and 29..37 stay: pages 0, 1 and 7, 8, 9
    assert (p.table[0] >= 0).tolist() == [True] * 2 + [False] * 5 + [True] * 3
    assert p.lens[0] == 38 and p.refs.sum() == 5


def test_compact():
    p = Pool(8, 2, 4, 4, [16], seed=3)
    p.fill_row(0, 9, [6, 1, 7])
    p.fill_row(1, 4, [3])
    p.table[1, 1] = 7  # behind the row's context: not an entry
    before = p.caches[0].copy()
    assert p.compact() == 4
    assert p.table[0, :3].tolist() == [0, 1, 2] and p.table[1, :2].tolist() == [3, 7]
    assert (p.caches[0][[0, 1, 2, 3]] == before[[6, 1, 7, 3]]).all()
    assert p.refs.tolist() == [1, 1, 1, 1, 0, 0, 0, 0]


@pytest.mark.parametrize("seed", range(20))
def test_random_walks_keep_the_counts(seed):
    p = Pool(40, 8, 6, 4, [8], seed=seed)
    r = np.random.RandomState(seed + 100)
    for _ in range(30):
        k = r.randint(4)
        if k == 0:
            row = r.randint(8)
            n = r.randint(0, 25)
            if p.lens[row] == 0 and (p.refs == 0).sum() >= p.blocks(n):
                p.fill_row(row, n)
        elif k == 1:
            p.fork(r.randint(0, 8, 3), r.randint(0, 8, 3))
        elif k == 2:
            p.free(r.randint(0, 8, 2), window=r.randint(0, 9), sinks=r.randint(0, 6))
        else:
            live = p.compact()
            assert (p.refs[:live] > 0).all() and (p.refs[live:] == 0).all()
        assert (counts(p) == p.refs).all()
        assert not p.err & REFS
