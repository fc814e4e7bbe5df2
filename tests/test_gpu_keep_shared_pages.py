"""dsa_cache_keep of rows that share pages: one that an entry would move to must be
the row's own, else the row stays as it is and DSA_DEVERR_REFS says so."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
P, PAGES, ROWS, COLS, REFS = 16, 60, 8, 12, 64


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import prep_token_gb300 as dp
    dp.library()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pool:
    """Rows of given lengths with pages of their own, and copies by dsa_cache_fork."""

    def __init__(self, lengths, forks=(), seed=0):
        import prep_token_gb300 as dp
        self.dp = dp
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.k = torch.randint(-999, 999, (PAGES, P, 2, 64), generator=g, device="cuda",
                               dtype=torch.int16)
        self.v = torch.randint(-999, 999, (PAGES, 2, P, 64), generator=g, device="cuda",
                               dtype=torch.int16).transpose(1, 2)
        r = np.random.RandomState(seed)
        order = r.permutation(PAGES)
        table, refs, lens = np.full((ROWS, COLS), -1), np.zeros(PAGES), np.zeros(ROWS)
        at = 0
        for row, n in enumerate(lengths):
            blocks = -(-n // P)
            table[row, :blocks] = order[at:at + blocks]
            refs[order[at:at + blocks]] = 1
            lens[row] = n
            at += blocks
        self.table, self.refs, self.lens = ints(table), ints(refs), ints(lens)
        self.err = ints([0])
        if forks:
            dp.dsa_cache_fork([self.k, self.v.transpose(1, 2)], self.refs, self.table, self.lens, P,
                              ints([a for a, _ in forks]), ints([b for _, b in forks]),
                              err_flags=self.err)
        assert int(self.err) == 0

    def row(self, row):
        """The row's entries in both caches."""
        n = int(self.lens[row])
        at = torch.arange(n, device="cuda")
        page = self.table[row].long()[at // P]
        return torch.cat([t[page, at % P].flatten(1) for t in (self.k, self.v)], 1)

    def state(self):
        return [t.clone() for t in (self.table, self.refs, self.lens, self.k, self.v)]

    def keep(self, rows, drafted, kept, caches=None):
        self.err.zero_()
        most = max([len(x) for x in kept] + [1])
        self.dp.dsa_cache_keep([self.k, self.v] if caches is None else caches, self.refs, self.table,
                               self.lens, P, ints(rows), ints(drafted),
                               ints([list(x) + [-1] * (most - len(x)) for x in kept]),
                               ints([len(x) for x in kept]), err_flags=self.err)
        return int(self.err)

    def counted(self):
        """page_refs are what the tables hold."""
        want = torch.zeros(PAGES, dtype=torch.int32)
        for row in range(ROWS):
            for e in self.table[row, :-(-int(self.lens[row]) // P)].tolist():
                want[e] += 1
        assert torch.equal(want, self.refs.cpu())


def unchanged(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("rows", [[0, 5], [5, 0], [0], [5]])
def test_forked_with_drafts_pending(rows):
    """64 drafts behind 10 tokens: four pages hold drafts and are both rows'."""
    for seed in range(10):
        p = Pool([74], [(0, 5)], seed)
        old = p.state()
        paths = {0: [1, 5, 20, 40, 63], 5: [3, 4, 17, 62]}
        assert p.keep(rows, [64] * len(rows), [paths[r] for r in rows]) == REFS
        assert unchanged(old, p.state())


def test_only_its_pages_are_refused():
    """Other rows of the list are carried out, and a row whose entries go to its own pages is
    whatever it shares in front of them."""
    p = Pool([74, 40, 42], [(0, 5), (2, 6)], 1)
    # 2 and 6 share two whole pages, 42 = 32 + 10 tokens: the last 8 drafts are in pages of their own
    want = {1: torch.cat([p.row(1)[:10], p.row(1)[[11, 15, 39]]]),
            2: torch.cat([p.row(2)[:34], p.row(2)[[35, 41]]]),
            6: torch.cat([p.row(6)[:34], p.row(6)[[34, 36]]])}
    same = {r: p.row(r) for r in (0, 5)}
    assert p.keep([1, 0, 2, 6], [30, 64, 8, 8], [[1, 5, 29], [7, 60], [1, 7], [0, 2]]) == REFS
    for row, rows in {**want, **same}.items():
        assert torch.equal(p.row(row), rows)
    p.counted()


def test_entries_that_stay_write_nothing():
    p = Pool([74], [(0, 5)], 2)
    want = {0: p.row(0)[:16], 5: p.row(5)[:10]}
    k, v = p.k.clone(), p.v.clone()
    assert p.keep([0, 5], [64, 64], [range(6), []]) == 0
    assert torch.equal(p.k, k) and torch.equal(p.v, v)
    for row, rows in want.items():
        assert torch.equal(p.row(row), rows)
    p.counted()


def test_a_page_given_back_in_the_same_call_is_still_shared():
    """The check sees the counts as they were before the call, in whatever order rows run."""
    for seed in range(20):
        p = Pool([74], [(0, 5)], seed)
        other = p.row(5)
        # row 0 gives back all but its first page; row 5 would write in the others only
        rows = [0, 5] if seed % 2 else [5, 0]
        path = list(range(6)) + [30, 50]
        lists = {0: range(6), 5: path}
        assert p.keep(rows, [64, 64], [lists[r] for r in rows]) == REFS
        assert int(p.lens[0]) == 16 and torch.equal(p.row(5), other)
        p.counted()
        # now they are its own
        want = torch.cat([other[:10], other[[10 + a for a in path]]])
        assert p.keep([5], [64], [path]) == 0
        assert torch.equal(p.row(5), want)
        p.counted()


def test_no_reference_at_all():
    """A page that counts as free is not the row's own either."""
    p = Pool([40], seed=3)
    p.refs[p.table[0, 0].long()] = 0
    old = p.state()
    assert p.keep([0], [30], [[4, 9]]) == REFS
    assert unchanged(old, p.state())


def test_without_caches_nothing_is_written():
    p = Pool([74], [(0, 5)], 4)
    assert p.keep([0, 5], [64, 64], [[1, 5], [2]], caches=[]) == 0
    assert p.lens[[0, 5]].tolist() == [12, 11]
    p.counted()


def test_long_lists_of_shared_pages():
    """The one entry that would go to a shared page is far behind in the list."""
    p = Pool([180], [(0, 5)], 5)
    old = p.state()
    path = list(range(150)) + [160, 170]  # only the last two move, to page 9 of 11
    assert p.keep([5], [180], [path]) == REFS
    assert unchanged(old, p.state())
    p.dp.dsa_cache_free(p.refs, p.table, p.lens, P, ints([0]), err_flags=p.err)
    want = p.row(5)[path]
    assert p.keep([5], [180], [path]) == 0
    assert torch.equal(p.row(5), want)
    p.counted()
