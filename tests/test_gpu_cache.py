"""Page upkeep on the GPU against the plain pool model: every table, count,
page byte and error bit has to be equal."""
import numpy as np
import pytest
import torch

from _pool import POOL, REFS, ROW, SLOT, Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import prep_token_gb300 as dp
    dp.library()


def ints(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


class Device:
    """The pool's arrays on the GPU, and the calls."""

    def __init__(self, p, extra_cols=0):
        import prep_token_gb300 as dp
        self.dp, self.P, self.N = dp, p.P, p.N
        self.caches = [torch.from_numpy(c).cuda() for c in p.caches]
        self.refs, self.lens = ints(p.refs), ints(p.lens)
        wide = torch.full((p.rows, p.cols + extra_cols), 7777, dtype=torch.int32, device="cuda")
        self.table = wide[:, :p.cols]
        self.table.copy_(ints(p.table))
        self.wide = wide
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def copy(self, src, dst):
        self.dp.dsa_cache_copy_pages(self.caches, self.N, ints(src), ints(dst), err_flags=self.err)

    def fork(self, parents, children):
        self.dp.dsa_cache_fork(self.caches, self.refs, self.table, self.lens, self.P,
                               ints(parents), ints(children), err_flags=self.err)

    def free(self, rows, window=0, sinks=0):
        self.dp.dsa_cache_free(self.refs, self.table, self.lens, self.P, ints(rows),
                               window=window, sinks=sinks, err_flags=self.err)

    def compact(self):
        return int(self.dp.dsa_cache_compact(self.caches, self.refs, self.table, self.lens,
                                             self.P, err_flags=self.err).item())

    def check(self, p):
        torch.cuda.synchronize()
        assert np.array_equal(self.refs.cpu().numpy(), p.refs)
        assert np.array_equal(self.table.cpu().numpy(), p.table)
        assert np.array_equal(self.lens.cpu().numpy(), p.lens)
        for got, want in zip(self.caches, p.caches):
            assert np.array_equal(got.cpu().numpy(), want)
        assert int(self.err.item()) == p.err
        assert (self.wide[:, p.cols:] == 7777).all()


# page bytes: the index-K page of 64 slots, one whose pages are not 16-byte
# aligned, one of a single word, one of more than two pieces of a copy
SIZES = [[8448], [132, 4, 2048], [70000, 528], [65536, 32768, 32764]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("n", [1, 7, 40])
def test_copy(sizes, n):
    p = Pool(100, 1, 1, 4, sizes, seed=n)
    d = Device(p)
    perm = np.random.RandomState(n).permutation(100)
    src, dst = perm[:n].copy(), perm[50:50 + n].copy()
    if n > 5:
        src[3] = dst[3]          # onto itself: nothing
        src[1], dst[2] = -1, 100  # outside the pool: left out
        src[4] = src[5]           # one source, two destinations
    d.copy(src, dst)
    p.copy(src, dst)
    assert p.err == (SLOT if n > 5 else 0)
    d.check(p)


def test_copy_of_nothing():
    p = Pool(4, 1, 1, 4, [64])
    d = Device(p)
    d.copy([], [])
    d.caches = []
    d.copy([0], [1])
    d.caches = [torch.from_numpy(c).cuda() for c in p.caches]
    d.check(p)


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("page", [1, 3, 64])
def test_fork_and_free(sizes, page):
    p = Pool(300, 40, 20, page, sizes, seed=page)
    for row, n in enumerate([0, 1, page, page + 1, 7 * page - 1, 20 * page]):
        p.fill_row(row, n)
    d = Device(p, extra_cols=3)
    parents = [4, 5, 0, 3, 3, 2, 1, 4, 4]
    children = [10, 11, 12, 13, 39, 20, 21, 22, 23]
    d.fork(parents, children)
    p.fork(parents, children)
    assert p.err == 0
    d.check(p)
    d.fork([22, 10], [30, 31])  # children of children
    p.fork([22, 10], [30, 31])
    d.check(p)
    d.free([10, 4, 39, 10, 0, 5])
    p.free([10, 4, 39, 10, 0, 5])
    assert p.err == 0
    d.check(p)


def test_fork_refusals_leave_no_trace():
    p = Pool(12, 10, 4, 4, [16])
    p.fill_row(0, 6)
    p.fill_row(1, 16)
    p.lens[2] = 17  # more blocks than the table has columns
    p.lens[3] = -1
    d = Device(p)
    parents = [0, 0, 0, 2, 3, -1, 10, 0, 0, 1, 0]
    children = [4, 4, 1, 5, 6, 7, 7, -1, 10, 8, 9]
    d.fork(parents, children)
    p.fork(parents, children)
    assert p.err == ROW and p.lens[4] == 6 and p.lens[8] == 16 and p.lens[7] == 0
    d.check(p)


def test_fork_gives_the_last_pages_in_order():
    p = Pool(6, 10, 2, 8, [32])
    p.fill_row(0, 11, [4, 1])
    d = Device(p)
    for q in (p, d):
        q.fork([0] * 6, [9, 8, 7, 6, 5, 4])
    assert p.err == POOL and (p.lens > 0).sum() == 5
    d.check(p)


def test_fork_skips_absent_and_bad_entries():
    p = Pool(20, 5, 8, 4, [16])
    p.fill_row(0, 30)
    p.free([0], window=9)
    p.fill_row(1, 6)
    p.table[1, 0] = 20
    p.fill_row(2, 7)
    p.table[2, 1] = -5
    d = Device(p)
    for q in (p, d):
        q.fork([0, 1, 2], [3, 4, 2])  # the last one's child is in use
    assert p.err == SLOT | ROW
    d.check(p)


def test_fork_from_a_large_pool_with_free_pages_far_up():
    p = Pool(70001, 70, 3, 4, [4], seed=5)
    p.refs[:] = 1
    p.refs[[69999, 70000, 33000, 16384]] = 0
    p.table[0, 0], p.lens[0] = 5, 3
    d = Device(p)
    for q in (p, d):
        q.fork([0] * 5, [1, 2, 3, 4, 5])
    assert p.table[1:5, 0].tolist() == [16384, 33000, 69999, 70000] and p.err == POOL
    d.check(p)


def test_fork_of_as_many_rows_as_a_call_takes():
    p = Pool(2100, 1100, 2, 4, [4], seed=6)
    p.fill_row(0, 5)
    d = Device(p)
    children = np.random.RandomState(0).permutation(np.arange(1, 1100))[:1024]
    for q in (p, d):
        q.fork([0] * 1024, children)
    assert p.err == 0
    d.check(p)


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 0), (64, 1), (63, 64), (65, 65), (300, 4),
                                          (10 ** 9, 0), (1, 10 ** 9), (100, 2 ** 31 - 1)])
def test_free_behind_a_window(window, sinks):
    p = Pool(100, 6, 12, 16, [64])
    for row, n in enumerate([0, 1, 16, 100, 191, 192]):
        p.fill_row(row, n)
    d = Device(p, extra_cols=1)
    for q in (p, d):
        q.free([3, 4, 5, 0, 1, 2, 5], window=window, sinks=sinks)
        q.free([4], window=max(1, window // 2), sinks=sinks // 2)
    assert p.err == 0
    d.check(p)


def test_free_errors():
    p = Pool(10, 4, 3, 4, [16])
    p.fill_row(0, 12)
    p.refs[p.table[0, 1]] = 0  # a page that nobody counts
    p.table[0, 2] = 10
    p.lens[1], p.lens[2] = 13, -3
    p.table[1] = [-1, -7, -1]
    d = Device(p)
    for q in (p, d):
        q.free([0, -1, 4, 1, 2])
    assert p.err == ROW | SLOT | REFS
    d.check(p)


@pytest.mark.parametrize("pages,live", [(1, 0), (1, 1), (31, 9), (64, 64), (65, 1), (1000, 300),
                                        (4096, 4000), (70001, 20000)])
def test_compact(pages, live):
    rows, page = 17, 4
    share = np.bincount(np.arange(live) % rows, minlength=rows)
    p = Pool(pages, rows, max(1, share.max() + 2), page, [16, 20], seed=live)
    for row in range(rows):
        if share[row]:
            p.fill_row(row, (share[row] - 1) * page + 1 + row % page)
    d = Device(p, extra_cols=2)
    before = [c.copy() for c in p.caches]
    table = p.table.copy()
    assert d.compact() == p.compact() == live
    d.check(p)
    for c, b in zip(p.caches, before):  # every entry still finds its own bytes
        held = table >= 0
        assert (c[p.table[held]] == b[table[held]]).all()
    assert d.compact() == live  # nothing more to move
    d.check(p)


def test_compact_follows_shared_pages_and_counts():
    p = Pool(50, 8, 6, 4, [8448, 4])
    p.fill_row(0, 22, [40, 3, 49, 7, 30, 31])
    p.fork([0, 0], [1, 2])
    p.free([1])
    d = Device(p)
    assert d.compact() == p.compact()
    assert p.err == 0
    d.check(p)


def test_compact_errors():
    p = Pool(30, 4, 3, 4, [16])
    p.fill_row(0, 12, [20, 21, 0])
    p.table[0, 1] = 30      # outside the pool
    p.fill_row(1, 5, [28, 29])
    p.refs[29] = 0          # nobody counts it
    p.lens[2], p.lens[3] = 13, -1
    d = Device(p)
    assert d.compact() == p.compact()
    assert p.err == ROW | SLOT | REFS
    d.check(p)


@pytest.mark.parametrize("seed", range(6))
def test_random_walks(seed):
    p = Pool(60, 9, 7, 4, [132 * 4, 36], seed=seed)
    for row in range(4):
        p.fill_row(row, p.rng.randint(1, 29))
    d = Device(p)
    r = np.random.RandomState(seed + 50)
    for _ in range(12):
        k = r.randint(3)
        a, b = r.randint(0, 9, 4), r.randint(0, 9, 4)
        w, s = r.randint(0, 20), r.randint(0, 9)
        for q in (p, d):
            if k == 0:
                q.fork(a, b)
            elif k == 1:
                q.free(a[:2], window=w, sinks=s)
            else:
                q.compact()
    d.check(p)


def test_on_another_stream_and_in_a_graph():
    """A captured fork, free and compact, replayed: the same as the model each time."""
    import prep_token_gb300 as dp
    p = Pool(64, 8, 6, 4, [64, 12], seed=1)
    p.fill_row(0, 18)
    p.fill_row(1, 7)
    d = Device(p)
    lists = [ints(x) for x in ([0, 1, 0], [5, 6, 7], [5, 0])]
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    live = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        dp.dsa_cache_fork(d.caches, d.refs, d.table, d.lens, 4, lists[0], lists[1], workspace=ws,
                          err_flags=d.err)
        dp.dsa_cache_free(d.refs, d.table, d.lens, 4, lists[2], err_flags=d.err)
        dp.dsa_cache_compact(d.caches, d.refs, d.table, d.lens, 4, live_pages=live, workspace=ws,
                             err_flags=d.err)

    def model():
        p.fork([0, 1, 0], [5, 6, 7])
        p.free([5, 0])
        p.compact()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    model()
    d.check(p)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        d.refs.copy_(ints(p.refs))
        g.replay()
        model()
        d.check(p)
        assert int(live.item()) == int((p.refs > 0).sum())


def test_binding_refusals():
    import prep_token_gb300 as dp
    p = Pool(4, 2, 2, 4, [16])
    d = Device(p)
    one = ints([0])
    with pytest.raises(ValueError, match="length"):
        dp.dsa_cache_copy_pages(d.caches, 4, one, ints([1, 2]))
    with pytest.raises(ValueError, match="pages of equal size"):
        dp.dsa_cache_copy_pages(d.caches, 3, one, one)
    with pytest.raises(ValueError, match="contiguous"):
        dp.dsa_cache_copy_pages([d.caches[0].t()], 4, one, one)
    with pytest.raises(TypeError, match="int32"):
        dp.dsa_cache_free(d.refs, d.table, d.lens, 4, one.long())
    with pytest.raises(dp.DsaError, match="DSA_ERR_SHAPE"):
        dp.dsa_cache_free(d.refs, d.table, d.lens, 4, one, window=-1)
    with pytest.raises(dp.DsaError, match="DSA_ERR_SHAPE"):
        dp.dsa_cache_fork(d.caches, d.refs, d.table, d.lens, 4, one, one,
                          workspace=torch.empty(4, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="fewer"):
        dp.dsa_cache_free(d.refs, d.table, d.lens[:1], 4, one)
    d.check(p)
