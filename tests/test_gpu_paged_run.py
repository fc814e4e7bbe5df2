"""A serving loop over one pool of pages: prompts stored, branches forked, old
pages behind a window freed, the pool packed, tokens appended -- and after each
step the attention of every live sequence and the indexer's logits against
plain caches that hold each sequence's own rows in order."""
import numpy as np
import pytest
import torch

import synth
from _attn import reference

pytestmark = pytest.mark.gpu
P, HKV, H, D, PAGES, ROWS, COLS = 64, 2, 8, 128, 60, 6, 16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import prep_token_gb300 as dp
    dp.library()


class Loop:
    """The pool on the GPU, and every sequence's K, V and index key rows as lists."""

    def __init__(self, seed):
        import prep_token_gb300 as dp
        self.dp = dp
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.k = torch.full((PAGES, P, HKV, D), float("nan"), **bf)
        self.v = torch.full((PAGES, P, HKV, D), float("nan"), **bf)
        self.index = torch.zeros(PAGES * P * 132, dtype=torch.uint8, device="cuda")
        self.refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
        self.table = torch.full((ROWS, COLS), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.own = {}  # row -> [k, v, index key] of its tokens
        inp = synth.make_tiny(seed=seed, T=4, H=8)
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.cos, self.sin, self.gamma, self.beta = map(up, (inp.cos, inp.sin, inp.gamma, inp.beta))
        self.inp = inp

    def caches(self):
        return [self.k, self.v, self.index]

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(torch.bfloat16)

    def append(self, row, n):
        """n tokens of a row: pages taken as they are needed, K, V and the indexer's
        key written to their slots."""
        have = int(self.lens[row])
        for j in range(-(-have // P), -(-(have + n) // P)):
            page = int((self.refs == 0).nonzero()[0])
            self.refs[page] = 1
            self.table[row, j] = page
        pos = torch.arange(have, have + n, device="cuda")
        slots = self.table[row].long()[pos // P] * P + pos % P
        k, v, ik = self.rand(n, HKV, D), self.rand(n, HKV, D), self.rand(n, D)
        self.k.view(-1, HKV, D)[slots], self.v.view(-1, HKV, D)[slots] = k, v
        self.dp.dsa_indexer_k_prepare_store(ik, pos, slots, self.cos, self.sin, self.gamma,
                                            self.beta, self.inp.eps, self.index, P,
                                            self.inp.rope_dim, self.inp.style, err_flags=self.err)
        self.lens[row] = have + n
        old = self.own.get(row)
        new = [k, v, ik]
        self.own[row] = new if old is None else [torch.cat(x) for x in zip(old, new)]

    def check(self, new, window=0, sinks=0):
        """new: {row: its last tokens that attend}, against each sequence alone."""
        rows = list(new)
        n = [new[r] for r in rows]
        q = self.rand(sum(n), H, D) * 2
        at = torch.tensor(rows, device="cuda")
        table, lens = self.table[at], self.lens[at]
        start = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device="cuda")
        out, lse = self.dp.dsa_paged_attention(q, self.k, self.v, table, start, lens, COLS * P,
                                               window=window, sinks=sinks, err_flags=self.err)
        # the plain caches: sequence b's rows in order, one "page" each
        most = max(self.own[r][0].shape[0] for r in rows)
        k = torch.zeros(len(rows), most, HKV, D, dtype=torch.bfloat16, device="cuda")
        v = torch.zeros_like(k)
        for b, r in enumerate(rows):
            m = self.own[r][0].shape[0]
            assert int(lens[b]) == m
            k[b, :m], v[b, :m] = self.own[r][0], self.own[r][1]
        one = torch.arange(len(rows), device="cuda", dtype=torch.int32)[:, None]
        want, z, tol, tol_l = reference(q, k, v, one, start, lens, D ** -0.5, window, sinks)
        assert ((out.double() - want).abs() <= tol).all()
        assert ((lse.double() - z).abs() <= tol_l).all()
        assert int(self.err.item()) == 0
        return rows, table, lens

    def check_index(self, rows, table, lens):
        """The logits of one query over each row equal those over its keys stored afresh."""
        q = torch.randint(0, 0x60, (len(rows), 16, D), generator=self.g, device="cuda").to(torch.uint8)
        w = torch.randn(len(rows), 16, generator=self.g, device="cuda")
        got = self.dp.dsa_indexer_mqa_logits(q, w, self.index, P, table, lens, COLS * P)
        fresh = torch.zeros(len(rows) * COLS * P * 132, dtype=torch.uint8, device="cuda")
        plain = torch.arange(len(rows) * COLS, device="cuda", dtype=torch.int32).view(-1, COLS)
        for b, r in enumerate(rows):
            ik = self.own[r][2]
            pos = torch.arange(ik.shape[0], device="cuda")
            self.dp.dsa_indexer_k_prepare_store(ik, pos, pos + b * COLS * P, self.cos, self.sin,
                                                self.gamma, self.beta, self.inp.eps, fresh, P,
                                                self.inp.rope_dim, self.inp.style)
        want = self.dp.dsa_indexer_mqa_logits(q, w, fresh, P, plain, lens, COLS * P)
        assert torch.equal(got, want)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("seed", [0, 1])
def test_serving_loop(seed):
    s = Loop(seed)
    dp = s.dp
    s.append(0, 300)
    s.append(1, 129)
    s.check_index(*s.check({0: 300, 1: 129}))              # prompts, whole
    dp.dsa_cache_fork(s.caches(), s.refs, s.table, s.lens, P, ints(0, 0, 1), ints(2, 3, 4),
                      err_flags=s.err)
    for child, parent in ((2, 0), (3, 0), (4, 1)):
        s.own[child] = list(s.own[parent])
    s.check_index(*s.check({r: 1 for r in range(5)}))
    for row, n in ((0, 1), (2, 70), (3, 1), (4, 200)):      # the branches part
        s.append(row, n)
    s.check_index(*s.check({0: 1, 2: 70, 3: 1, 1: 1, 4: 200}))
    dp.dsa_cache_free(s.refs, s.table, s.lens, P, ints(0, 1), err_flags=s.err)
    del s.own[0], s.own[1]
    live = dp.dsa_cache_compact(s.caches(), s.refs, s.table, s.lens, P, err_flags=s.err)
    assert int(live) == int((s.refs > 0).sum()) == int(s.refs.nonzero().max()) + 1
    s.check_index(*s.check({2: 5, 3: 1, 4: 1}))
    s.append(3, 64)
    s.append(0, 10)                                        # a freed row serves again
    s.check_index(*s.check({0: 10, 2: 1, 3: 64, 4: 1}))
    # sliding-window layers: what the window has left behind goes back to the pool
    before = int((s.refs > 0).sum())
    s.check({2: 1, 3: 1, 4: 1}, window=100, sinks=4)
    dp.dsa_cache_free(s.refs, s.table, s.lens, P, ints(2, 3, 4), window=100, sinks=4,
                      err_flags=s.err)
    assert int((s.refs > 0).sum()) < before
    s.check({2: 1, 3: 1, 4: 1}, window=100, sinks=4)
    dp.dsa_cache_compact(s.caches(), s.refs, s.table, s.lens, P, err_flags=s.err)
    for row in (2, 3, 4):
        s.append(row, 1)
    s.check({2: 1, 3: 1, 4: 1}, window=100, sinks=4)
    s.check({4: 1, 2: 1}, window=60)


def test_prepared_call():
    from _attn import Batch
    b = Batch([1, 7], [600, 90], H, HKV, seed=30)
    import prep_token_gb300 as dp
    call = dp.prepare_paged_attention(b.q, b.k, b.v, b.table, b.start, b.lens, 600)
    out, lse = call()
    b.check(out, lse)
    b.q.neg_()
    assert call()[0] is out
    b.check(out, lse)
    with pytest.raises(dp.DsaError, match="SHAPE"):
        dp.prepare_paged_attention(b.q, b.k, b.v, b.table, b.start, b.lens, 600, window=-1)()
