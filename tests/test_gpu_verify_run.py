"""A loop that drafts and verifies over one pool of pages: norm, projection, append
of the drafts' K, V and indexer keys, attention over their trees, the accepted
ones kept -- with branches forked, rows freed and the pool packed between -- and
after each step every cache against plain lists of each sequence's own rows."""
import numpy as np
import pytest
import torch

import synth
from _tree import random_tree, reference, words_of

pytestmark = pytest.mark.gpu
P, HKV, H, D, PAGES, ROWS, COLS, N = 16, 2, 8, 128, 120, 6, 40, 512


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import prep_token_gb300 as dp
    dp.library()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Loop:
    def __init__(self, seed):
        import prep_token_gb300 as dp
        self.dp = dp
        self.r = np.random.RandomState(seed)
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.k = torch.full((PAGES, P, HKV, D), float("nan"), **bf)
        self.v = torch.full((PAGES, HKV, P, D), float("nan"), **bf).transpose(1, 2)  # heads before tokens
        self.index = torch.zeros(PAGES * P * 132, dtype=torch.uint8, device="cuda")
        self.refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
        self.table = torch.full((ROWS, COLS), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        inp = synth.make_tiny(seed=seed, T=4, H=8)
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.cos, self.sin, self.gamma, self.beta = map(up, (inp.cos, inp.sin, inp.gamma, inp.beta))
        self.eps, self.style, self.rope = inp.eps, inp.style, inp.rope_dim
        rand = lambda *s: torch.randn(*s, generator=self.g, device="cuda")  # noqa: E731
        self.rand = rand
        self.weight = (rand(N, (H + 2 * HKV) * D + D) * N ** -0.5).bfloat16()
        self.norm = torch.rand(N, generator=self.g, device="cuda") + 0.5
        self.qk = torch.rand(2, D, generator=self.g, device="cuda") + 0.5
        self.views = dp.TokenViews([self.k, self.v, *dp.index_k_token_views(self.index, P)])
        self.pages = [self.k, self.v.transpose(1, 2), self.index]  # as the bytes that they are
        self.own = {}  # row -> [k, v, codes, scales] of its tokens

    def entries(self, row, tokens):
        """What the caches hold for these tokens of a row."""
        page, at = self.table[row].long()[tokens // P], tokens % P
        return [t[page, at].clone() for t in self.views.caches]

    def draft(self, drafts, window=0, sinks=0):
        """drafts: {row: number}; a random tree for each.  Returns the trees' bits."""
        rows = list(drafts)
        trees, slots, depth = {}, [], []
        for row in rows:
            n, have = drafts[row], int(self.lens[row])
            trees[row] = random_tree(n, self.r)
            for j in range(-(-have // P), -(-(have + n) // P)):
                page = int((self.refs == 0).nonzero()[0])
                self.refs[page] = 1
                self.table[row, j] = page
            at = torch.arange(have, have + n, device="cuda")
            slots.append(self.table[row].long()[at // P] * P + at % P)
            depth += [have + bin(bits).count("1") - 1 for bits in trees[row]]
            self.lens[row] = have + n
        T = sum(drafts.values())
        slots, positions = torch.cat(slots), torch.tensor(depth, device="cuda")
        x, res = self.rand(T, N).bfloat16(), (self.rand(T, N) * 2).bfloat16()
        y, res = self.dp.dsa_rms_norm(x, self.norm, 1e-6, residual=res)
        qkv = y @ self.weight
        q, k, v, ik = qkv.split([H * D, HKV * D, HKV * D, D], 1)
        q, k, v = (t.unflatten(1, (-1, D)) for t in (q, k, v))
        q = self.dp.dsa_kv_append(q, k, v, positions, slots, self.cos, self.sin, self.k, self.v,
                                  rope_dim=self.rope, rope_style=self.style, q_gamma=self.qk[0],
                                  k_gamma=self.qk[1], err_flags=self.err)
        self.dp.dsa_indexer_k_prepare_store(ik, positions, slots, self.cos, self.sin, self.gamma,
                                            self.beta, self.eps, self.index, P, self.rope,
                                            self.style, err_flags=self.err)
        # every row's caches: its own rows in order, then the drafts
        most = max(int(self.lens[r]) for r in rows)
        kk = torch.zeros(len(rows), most, HKV, D, dtype=torch.bfloat16, device="cuda")
        vv = torch.zeros_like(kk)
        at = 0
        for b, row in enumerate(rows):
            have, n = int(self.lens[row]) - drafts[row], drafts[row]
            if have:
                kk[b, :have], vv[b, :have] = self.own[row][0], self.own[row][1]
            new = self.entries(row, torch.arange(have, have + n, device="cuda"))
            assert torch.equal(new[1], v[at:at + n])
            kk[b, have:have + n], vv[b, have:have + n] = new[0], new[1]
            at += n
        start = ints([0] + list(np.cumsum([drafts[r] for r in rows])))
        table, lens = self.table[ints(rows).long()], self.lens[ints(rows).long()]
        words = -(-max(drafts.values()) // 32)
        mask = words_of([bits for r in rows for bits in trees[r]], words)
        out, lse = self.dp.dsa_tree_attention(q, self.k, self.v, table, start, lens, COLS * P, mask,
                                              window=window, sinks=sinks, err_flags=self.err)
        one = torch.arange(len(rows), device="cuda", dtype=torch.int32)[:, None]
        want, z, tol, tol_l = reference(q, kk, vv, one, start, lens, mask, D ** -0.5, window, sinks)
        assert ((out.double() - want).abs() <= tol).all()
        assert ((lse.double() - z).abs() <= tol_l).all()
        return trees

    def keep(self, drafts, trees):
        """A random path of each tree is accepted, of any length."""
        kept = []
        for row in drafts:
            tip = int(self.r.randint(-1, drafts[row]))
            path = [j for j in range(drafts[row]) if tip >= 0 and trees[row][tip] >> j & 1]
            have = int(self.lens[row]) - drafts[row]
            new = self.entries(row, have + torch.tensor(path, dtype=torch.long, device="cuda"))
            old = self.own.get(row) or [t[:0] for t in new]
            self.own[row] = [torch.cat(x) for x in zip(old, new)]
            kept.append(path)
        most = max([len(p) for p in kept] + [1])
        self.dp.dsa_cache_keep(self.views, self.refs, self.table, self.lens, P, ints(list(drafts)),
                               ints([drafts[r] for r in drafts]),
                               ints([p + [9] * (most - len(p)) for p in kept]),
                               ints([len(p) for p in kept]), err_flags=self.err)
        self.check()

    def check(self):
        assert int(self.err) == 0
        counts = torch.zeros_like(self.refs)
        for row in range(ROWS):
            n = int(self.lens[row])
            assert n == (self.own[row][0].shape[0] if row in self.own else 0)
            used = self.table[row, :-(-n // P)].long()
            counts.index_add_(0, used, torch.ones_like(used, dtype=torch.int32))
            if n:
                for got, want in zip(self.entries(row, torch.arange(n, device="cuda")), self.own[row]):
                    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
        assert torch.equal(counts, self.refs)

    def step(self, drafts, **kw):
        self.keep(drafts, self.draft(drafts, **kw))


@pytest.mark.parametrize("seed", range(3))
def test_drafting_loop(seed):
    s = Loop(seed)
    s.step({0: 40, 1: 70, 2: 1})
    s.step({0: 8, 1: 8, 2: 8})
    for _ in range(3):
        s.step({r: int(s.r.randint(1, 50)) for r in (0, 1, 2)})
    if int(s.lens[1]):
        s.dp.dsa_cache_fork(s.pages, s.refs, s.table, s.lens, P, ints([1]), ints([4]),
                            err_flags=s.err)
        s.own[4] = list(s.own[1])
        s.check()
        s.step({1: 12, 4: 30, 0: 5}, window=40, sinks=3)
    s.dp.dsa_cache_free(s.refs, s.table, s.lens, P, ints([0]), err_flags=s.err)
    del s.own[0]
    s.dp.dsa_cache_compact(s.pages, s.refs, s.table, s.lens, P, err_flags=s.err)
    s.check()
    s.step({1: 33, 0: 20, 2: 7})
    s.step({1: 3, 0: 64, 2: 32}, window=17)
