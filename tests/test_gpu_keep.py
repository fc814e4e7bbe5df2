"""dsa_cache_keep against a plain model on the host: every byte of every cache,
every table and count."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ROW, SLOT, REFS = 16, 2, 64


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import prep_token_gb300 as dp
    dp.library()


class Pool:
    """Rows of drafts over a shuffled pool; caches as tensors with one or two dimensions
    behind [pages, page], views of whatever strides."""

    def __init__(self, before, drafted, kept, page=16, shapes=((4, 64),), dtype=torch.int16,
                 views=None, seed=0, spare_rows=2):
        r = np.random.RandomState(seed)
        n = len(before)
        rows = n + spare_rows
        self.page = page
        length = np.zeros(rows, np.int32)
        self.which = r.permutation(rows)[:n].astype(np.int32)
        for i, row in enumerate(self.which):
            length[row] = before[i] + drafted[i]
        blocks = -(-length // page)
        cols = int(blocks.max(initial=0)) + 2
        pages = int(blocks.sum()) + 3
        perm = r.permutation(pages)
        self.table = r.choice([-1, 0, 7, 2 ** 30], (rows, cols)).astype(np.int32)  # past a row's end
        self.refs = np.zeros(pages, np.int32)
        at = 0
        for row in range(rows):
            self.table[row, :blocks[row]] = perm[at:at + blocks[row]]
            self.refs[perm[at:at + blocks[row]]] = 1
            at += blocks[row]
        self.lens, self.drafted = length, np.array(drafted, np.int32)
        most = max([len(k) for k in kept] + [1])
        self.kept = np.full((n, most), -7, np.int32)
        for i, k in enumerate(kept):
            self.kept[i, :len(k)] = k
        self.n_kept = np.array([len(k) for k in kept], np.int32)
        g = torch.Generator(device="cuda").manual_seed(seed)
        if views is None:
            self.store = [torch.randint(-30000, 30000, (pages, page, *s), generator=g, device="cuda",
                                        dtype=dtype) for s in shapes]
            self.views = self.store
        else:
            self.store, self.views = views(pages, page, g)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def model(self, caches):
        """The same on the host, entry by entry; returns the error bits."""
        err, seen, P = 0, set(), self.page
        for i, row in enumerate(self.which.tolist()):
            d, k = int(self.drafted[i]), int(self.n_kept[i])
            again = row in seen
            seen.add(row)
            if again or not 0 <= row < len(self.lens) or not 0 <= k <= min(d, self.kept.shape[1]):
                err |= ROW
                continue
            L = int(self.lens[row])
            list_ = self.kept[i, :k].tolist()
            if L < d or -(-L // P) > self.table.shape[1] or sorted(set(list_)) != list_ \
                    or (list_ and (list_[0] < 0 or list_[-1] >= d)):
                err |= ROW
                continue
            before = L - d
            for j, a in enumerate(list_):
                if a == j:
                    continue
                f, t = self.table[row, (before + a) // P], self.table[row, (before + j) // P]
                if not (0 <= f < len(self.refs) and 0 <= t < len(self.refs)):
                    err |= SLOT
                    continue
                for c in caches:
                    c[t, (before + j) % P] = c[f, (before + a) % P]
            for b in range(-(-(before + k) // P), -(-L // P)):
                e = int(self.table[row, b])
                if e < 0:
                    continue
                self.table[row, b] = -1
                if e >= len(self.refs):
                    err |= SLOT
                elif self.refs[e] <= 0:
                    err |= REFS
                else:
                    self.refs[e] -= 1
            self.lens[row] = before + k
        return err

    def device(self):
        up = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        return [up(x) for x in (self.refs, self.table, self.lens, self.which, self.drafted, self.kept,
                                self.n_kept)]

    def check(self, caches=None):
        import prep_token_gb300 as dp
        refs, table, lens, which, drafted, kept, n_kept = self.device()
        want = [v.cpu().clone() for v in self.views]
        outside = [s.clone() for s in self.store]
        dp.dsa_cache_keep(self.views if caches is None else caches, refs, table, lens, self.page,
                          which, drafted, kept, n_kept, err_flags=self.err)
        err = self.model([w.numpy() if w.dtype != torch.bfloat16 else w.view(torch.int16).numpy()
                          for w in want])
        assert int(self.err) == err
        for v, w, s, o in zip(self.views, want, self.store, outside):
            assert torch.equal(v.cpu(), w)
            v.copy_(w)
            o_view = o.as_strided(v.shape, v.stride(), v.storage_offset()) \
                if v.dtype == o.dtype else None
            if o_view is not None:  # nothing else in the store has changed
                o_view.copy_(w)
                assert torch.equal(s, o)
        for got, now in ((refs, self.refs), (table, self.table), (lens, self.lens)):
            assert np.array_equal(got.cpu().numpy(), now)
        return err


def random_case(n, r, most_before=100, most_drafts=40):
    before = r.randint(0, most_before, n)
    drafted = r.randint(0, most_drafts + 1, n)
    kept = [np.sort(r.choice(d, r.randint(0, d + 1), replace=False)) if d else [] for d in drafted]
    return before, drafted, kept


@pytest.mark.parametrize("page", [1, 3, 8, 16, 64])
@pytest.mark.parametrize("shapes", [((4, 64),), ((128,), (4,)), ((1, 2), (8, 128), (3, 6)), ((66,),)])
def test_random(page, shapes):
    for seed in range(4):
        r = np.random.RandomState(seed)
        n = [1, 5, 17, 40][seed]
        assert Pool(*random_case(n, r), page=page, shapes=shapes, seed=seed).check() == 0


def test_nothing_and_everything_kept():
    before, drafted = [0, 0, 10, 16, 30, 5], [8, 8, 6, 16, 34, 0]
    assert Pool(before, drafted, [[], range(8), [], range(16), [], []]).check() == 0
    assert Pool(before, drafted, [[7], [0], [5], [15], [33], []], page=8).check() == 0


def test_long_lists():
    r = np.random.RandomState(1)
    kept = [np.sort(r.choice(500, k, replace=False)) for k in (130, 300, 129, 1)]
    kept[2] = np.concatenate([np.arange(128), [400]])
    assert Pool([3, 60, 0, 9], [500] * 4, kept, page=16, shapes=((2, 32), (40,))).check() == 0


def strided(pages, page, g):
    store = [torch.randint(-99, 99, (pages, 3, page, 2, 72), generator=g, device="cuda",
                           dtype=torch.int16),
             torch.randint(-99, 99, (pages, page, 80), generator=g, device="cuda", dtype=torch.int16),
             torch.randint(-99, 99, (page, pages, 2, 64), generator=g, device="cuda",
                           dtype=torch.int16)]
    views = [store[0].transpose(1, 2)[..., 0, :64], store[1][..., 6:72],
             store[2].permute(1, 0, 2, 3)]
    return store, views


@pytest.mark.parametrize("page", [4, 16, 33])
def test_strided_views(page):
    r = np.random.RandomState(page)
    assert Pool(*random_case(9, r), page=page, views=strided, seed=page).check() == 0


@pytest.mark.parametrize("layout", ["paged", "token_major"])
def test_index_k_cache(layout):
    import prep_token_gb300 as dp

    def views(pages, page, g):
        flat = torch.randint(0, 256, (pages * page * 132,), generator=g, device="cuda",
                             dtype=torch.uint8)
        return [flat] * 2, dp.index_k_token_views(flat, page, layout)

    p = Pool(*random_case(11, np.random.RandomState(2)), page=16, views=views)
    codes, scales = dp.cache_views(p.store[0], 16)
    n_views = len(p.views)
    assert n_views == (2 if layout == "paged" else 1)
    if layout == "paged":
        assert torch.equal(p.views[0].reshape(-1, 128), codes)
        assert torch.equal(p.views[1].reshape(-1, 4).view(torch.float32).view(-1).view(torch.int32),
                           scales.view(torch.int32))
    p.store = p.store[:1] * n_views
    refs, table, lens, which, drafted, kept, n_kept = p.device()
    want = [v.cpu().clone() for v in p.views]
    dp.dsa_cache_keep(dp.TokenViews(p.views), refs, table, lens, 16, which, drafted, kept, n_kept)
    p.model([w.numpy() for w in want])
    for v, w in zip(p.views, want):
        assert torch.equal(v.cpu(), w)


def test_many_views():
    p = Pool(*random_case(6, np.random.RandomState(4)), shapes=((2, 64),) * 256, page=8)
    assert p.check() == 0


@pytest.mark.parametrize("usual", [True, False])
@pytest.mark.parametrize("order", ["expanded", "sliced", "overlapping"])
def test_lists_of_other_strides(order, usual):
    """One list for all rows by expand, lists out of wider rows; rows that overlap are refused."""
    import prep_token_gb300 as dp
    n = 40
    p = Pool([7 * i for i in range(n)], [12] * n, [[1, 2, 5, 11]] * n, seed=1, shapes=((4, 64), (8,)))
    d = p.device()
    if order == "expanded":
        d[5] = d[5][:1].clone().expand(n, -1)
    elif order == "sliced":
        wide = torch.full((n, 9), -3, dtype=torch.int32, device="cuda")
        wide[:, 2:6] = d[5]
        d[5] = wide[:, 2:6]
    else:
        d[5] = d[5].flatten().as_strided((n, 4), (2, 1))
    want = [v.cpu().clone() for v in p.views]
    call = lambda: dp.dsa_cache_keep(  # noqa: E731
        p.views, *d[:3], p.page, *d[3:], err_flags=p.err,
        stream=None if usual else torch.cuda.current_stream())
    if order == "overlapping":
        with pytest.raises(dp.DsaError, match="SHAPE"):
            call()
        return
    call()
    assert int(p.err) == p.model([w.numpy() for w in want]) == 0
    assert all(torch.equal(v.cpu(), w) for v, w in zip(p.views, want))
    assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(d[:3], (p.refs, p.table, p.lens)))


def test_without_caches():
    p = Pool(*random_case(6, np.random.RandomState(5)), shapes=())
    assert p.check() == 0


def test_entries_that_may_not_be_carried_out():
    before, drafted = [10] * 12, [20] * 12
    kept = [[1, 5, 7]] * 12
    p = Pool(before, drafted, kept, seed=3)
    p.which[1] = -1
    p.which[2] = len(p.lens)
    p.which[3] = p.which[0]            # named before
    p.drafted[4] = 31                  # more than the row has
    p.kept[5] = [5, 5, 7]
    p.kept[6] = [7, 5, 9]
    p.kept[7] = [-1, 2, 3]
    p.kept[8] = [1, 2, 20]
    p.n_kept[9] = 4                    # more than the list holds
    p.drafted[10], p.n_kept[10] = 2, 3
    assert p.check() == ROW
    p = Pool(before, drafted, kept, seed=4)
    p.lens[p.which[2]] = 5000          # longer than the table
    p.n_kept[3] = -1
    p.drafted[5] = -2
    assert p.check() == ROW


def test_bad_pages_and_counts():
    p = Pool([10, 10, 10, 40], [30, 30, 30, 30], [[1, 5, 20]] * 3 + [[]], seed=5)
    a, b, c, d = p.which
    p.table[a, 10 // 16] = -1          # where the first ones go
    p.table[b, 30 // 16] = len(p.refs)  # where the last one is
    p.refs[p.table[d, 3]] = 0
    assert p.check() == SLOT | REFS


def test_captured():
    import prep_token_gb300 as dp
    p = Pool(*random_case(8, np.random.RandomState(6)), shapes=((4, 64), (8,)))
    state = p.device()
    now = [x.clone() for x in state]
    first = [v.clone() for v in p.views]
    views = dp.TokenViews(p.views)
    dp.dsa_cache_keep(views, *now[:3], p.page, *now[3:])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dp.dsa_cache_keep(views, *now[:3], p.page, *now[3:])
    for _ in range(2):
        for a, b in zip(now, state):
            a.copy_(b)
        for a, b in zip(p.views, first):
            a.copy_(b)
        graph.replay()
    want = [v.cpu().clone() for v in first]
    p.model([w.numpy() for w in want])
    assert all(torch.equal(v.cpu(), w) for v, w in zip(p.views, want))
    assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(now, (p.refs, p.table, p.lens)))


def test_two_pools_at_once():
    """Calls on two streams, each with a pool and a workspace of its own."""
    import prep_token_gb300 as dp
    pools = [Pool(*random_case(30, np.random.RandomState(20 + i)), seed=i, page=8) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in pools]
    state = [p.device() for p in pools]
    want = [[v.cpu().clone() for v in p.views] for p in pools]
    torch.cuda.synchronize()
    for p, d, s in zip(pools, state, streams):
        with torch.cuda.stream(s):
            dp.dsa_cache_keep(p.views, *d[:3], p.page, *d[3:])
    torch.cuda.synchronize()
    for p, d, w in zip(pools, state, want):
        p.model([x.numpy() for x in w])
        assert all(torch.equal(v.cpu(), x) for v, x in zip(p.views, w))
        assert all(np.array_equal(g.cpu().numpy(), x) for g, x in zip(d, (p.refs, p.table, p.lens)))


def test_on_another_stream():
    import prep_token_gb300 as dp
    p = Pool(*random_case(8, np.random.RandomState(7)))
    d = p.device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = [v.cpu().clone() for v in p.views]
    dp.dsa_cache_keep(p.views, *d[:3], p.page, *d[3:], stream=side)
    side.synchronize()
    p.model([w.numpy() for w in want])
    assert torch.equal(p.views[0].cpu(), want[0])
