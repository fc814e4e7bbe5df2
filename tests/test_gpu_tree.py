"""dsa_tree_attention against its definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

from _attn import Batch
from _tree import Trees, words_of

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import prep_token_gb300 as dp
    dp.library()


def go(*args, **kw):
    b = Trees(*args, **kw)
    b.check(*b.run())
    assert int(b.err) == 0
    return b


HEADS = [(64, 8, 128), (8, 8, 64), (5, 1, 128), (128, 1, 64), (32, 4, 64), (1, 1, 128)]


@pytest.mark.parametrize("heads,kv,dim", HEADS)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("masks", ["tree", "any", "chain"])
def test_heads(heads, kv, dim, dtype, masks):
    go([5, 1, 0, 33, 64], [300, 1, 0, 700, 64], heads, kv, dim, dtype=dtype, masks=masks,
       seed=heads + dim)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 192])
@pytest.mark.parametrize("masks", ["tree", "any"])
def test_pages(page, masks):
    go([7, 40, 3], [130, 513, 1000], 16, 2, 128, page=page, masks=masks, seed=page)


@pytest.mark.parametrize("ctx", [1, 2, 31, 32, 33, 63, 127, 128, 129, 160, 255, 256, 257, 384, 1025])
def test_lengths(ctx):
    """Drafts that start and end anywhere in a block of keys, up to the whole context."""
    n = [1, min(ctx, 8), min(ctx, 31), min(ctx, 32), min(ctx, 33), min(ctx, 65), min(ctx, 130)]
    go(n, [ctx] * len(n), 8, 2, 128, page=16, masks="any", seed=ctx)
    go(n, [ctx] * len(n), 8, 2, 64, page=64, seed=ctx)


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (17, 0), (64, 4), (100, 130), (128, 0),
                                          (1000, 16), (5000, 3)])
@pytest.mark.parametrize("masks", ["tree", "any", "chain"])
def test_windows(window, sinks, masks):
    go([5, 1, 33, 64, 20], [300, 700, 900, 64, 2000], 16, 4, 128, page=16, masks=masks,
       window=window, sinks=sinks, seed=window)
    go([9, 60], [4000, 1300], 8, 1, 64, masks=masks, window=window, sinks=sinks, seed=sinks)


@pytest.mark.parametrize("n,words", [(300, 10), (300, 4), (64, 1), (40, 5), (12, 0)])
def test_mask_words(n, words):
    """Trees of many words, drafts past the words, and words past the drafts."""
    b = go([n, 3], [n + 200, 90], 8, 2, 128, masks="any", words=words, seed=n)
    c = Trees([n, 3], [n + 200, 90], 8, 2, 128, masks="any", words=words, seed=n)
    if words:  # a mask of wider rows
        wide = torch.full((c.mask.shape[0], words + 3), -1, dtype=torch.int32, device="cuda")
        wide[:, 1:1 + words] = c.mask
        c.mask = wide[:, 1:1 + words]
        assert torch.equal(c.run()[0], b.run()[0])


def test_long_contexts_are_cut_and_joined():
    for masks in ("tree", "any"):
        go([60, 8], [9000, 20000], 16, 2, 128, masks=masks, poison=False, seed=1)
        go([16, 1], [30000, 5], 8, 1, 64, masks=masks, poison=False, seed=2)


@pytest.mark.parametrize("window,sinks", [(0, 0), (5000, 300)])
def test_tiles_that_go_round(window, sinks):
    """Several tiles of a sequence over long contexts, each from a key block of its own on."""
    go([200, 3, 90], [17000, 200, 9001], 8, 1, 128, masks="any", window=window, sinks=sinks, seed=1)
    go([130, 128], [20000, 12345], 16, 2, 64, masks="tree", window=window, sinks=sinks, seed=2)
    go([70], [70 + 128 * 300], 8, 1, 64, masks="any", window=window, sinks=sinks, poison=False, seed=3)


@pytest.mark.parametrize("batch,dim", [(33, 128), (70, 64), (100, 128)])
def test_many_sequences_cut(batch, dim):
    """More sequences than a warp has lanes, idle ones and unequal ones among them."""
    r = np.random.RandomState(batch)
    n = r.randint(0, 9, batch) * (r.rand(batch) < 0.8)
    ctx = np.where(n > 0, n + r.randint(0, 3000, batch), 0)
    ctx[batch // 2], n[batch // 2] = 9000, 8
    go(n.tolist(), ctx.tolist(), 8, 2, dim, page=16, seed=batch, poison=dim == 64)


def test_whole_items():
    go([20] * 100, [150] * 100, 32, 8, 64, page=16, seed=3)
    go([64] * 60, list(range(64, 124)), 32, 8, 128, seed=4)


def test_chain_is_causal():
    """A chain's mask gives what dsa_paged_attention gives, within the same bounds."""
    t = Trees([40, 7], [700, 90], 16, 2, masks="chain", seed=5)
    b = Batch([40, 7], [700, 90], 16, 2, seed=5)
    for name in ("q", "k", "v", "table", "start", "lens"):
        setattr(t, name, getattr(b, name))
    out, lse = t.run()
    t.check(out, lse)
    b.check(out, lse)


def test_rows_that_see_nothing():
    t = Trees([6, 4], [6, 4], 8, 2, masks="tree", seed=6)  # nothing before the drafts
    t.mask[2] = 0
    t.mask[7] = 1 << 10  # behind the drafts
    out, lse = t.run()
    t.check(out, lse)
    assert (out[[2, 7]] == 0).all() and torch.isneginf(lse[[2, 7]]).all()


def test_more_drafts_than_context():
    """A context shorter than its drafts: the first of them have no key."""
    t = Trees([20, 5], [20, 50], 8, 2, masks="any", seed=7, poison=False)
    t.lens[0] = 12
    t.check(*t.run())
    t = Trees([20, 5], [20, 50], 8, 2, masks="tree", seed=8, poison=False, window=6)
    t.lens[0] = 0
    t.check(*t.run())


def test_context_longer_than_max_context():
    t = Trees([5, 40], [500, 333], 8, 2, masks="any", seed=9, max_context=400, poison=False)
    t.check(*t.run())


def test_values_that_are_not_finite():
    """A draft whose value is not finite spoils the rows that see it, their lse not; one that
    nobody sees spoils nothing (the pools are poisoned)."""
    t = Trees([12], [150], 8, 2, masks="tree", seed=10)
    before = 138
    page, off = int(t.table[0, (before + 3) // 64]), (before + 3) % 64
    want, z = t.run()
    t.v[page, off, 0, 5] = math.inf
    out, lse = t.run()
    sees = (t.mask[:, 0] >> 3 & 1).bool()
    assert sees.any() and not sees.all()
    assert torch.equal(lse, z)
    assert (~torch.isfinite(out[sees][:, :4, 5])).all()
    assert torch.equal(out[~sees], want[~sees]) and torch.equal(out[:, 4:], want[:, 4:])
    t.v[page, off, 0, 5] = 0
    t.k[page, off, 1, 7] = math.nan
    out, lse = t.run()
    assert torch.isnan(lse[sees][:, 4:]).all() and torch.isfinite(lse[~sees]).all()
    assert torch.isfinite(lse[:, :4]).all() and torch.isfinite(out[~sees]).all()


def test_bad_pages():
    t = Trees([9, 4], [200, 300], 8, 2, masks="tree", seed=11, page=16)
    t.table[0, 2], t.table[1, (300 - 4) // 16] = -1, t.k.shape[0]
    out, lse = t.run()
    t.check(out, lse)
    assert int(t.err) == 2 and torch.isnan(out[:9]).all()


def test_rows_behind_the_last_sequence():
    t = Trees([5, 3], [100, 60], 8, 2, masks="any", seed=12, extra_rows=4)
    out, lse = torch.full_like(t.q, 7.0), torch.full((12, 8), 7.0, device="cuda")
    t.run(out=out, lse=lse)
    t.check(out, lse)
    assert (out[8:] == 7).all() and (lse[8:] == 7).all()


def test_captured_graphs_and_streams():
    import prep_token_gb300 as dp
    t = Trees([60, 1, 20], [3000, 50, 800], 16, 2, masks="tree", seed=13)
    u = Trees([60, 1, 20], [3000, 50, 800], 16, 2, masks="any", seed=14)
    ws = torch.empty(dp.dsa_paged_attention_max_workspace_bytes(128), dtype=torch.uint8,
                     device="cuda")
    out, lse = t.run(workspace=ws)
    t.check(out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.run(out=out, lse=lse, workspace=ws, pdl=True)
        second = t.run(workspace=ws, pdl=True)
    for name in ("q", "k", "v", "table", "mask"):
        getattr(t, name).copy_(getattr(u, name)) if getattr(t, name).shape == \
            getattr(u, name).shape else None
    graph.replay()
    t.check(out, lse)
    assert torch.equal(second[0], out) and torch.equal(second[1], lse)
    call = dp.prepare_tree_attention(t.q, t.k, t.v, t.table, t.start, t.lens, t.max_context, t.mask)
    got = call()
    assert torch.equal(got[0], out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = t.run(stream=side)
    side.synchronize()
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)


def test_same_results_again():
    t = Trees([60, 16, 3], [5000, 700, 12000], 32, 4, masks="tree", seed=15, poison=False)
    out, lse = t.run()
    for _ in range(10):
        again = t.run()
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("n", [1, 33, 128])
def test_each_bit(n):
    """Equal scores and values one-hot by draft: out says which drafts a row sees."""
    t = Trees([n], [n + 50], 2, 1, masks="any", seed=n, poison=False)
    t.q.zero_()
    t.v.zero_()
    before = 50
    for j in range(n):
        key = before + j
        t.v[int(t.table[0, key // 64]), key % 64, 0, j % 128] = 1
    out, lse = t.run()
    bits = np.unpackbits(t.mask.cpu().numpy().view(np.uint8), axis=1, bitorder="little")[:, :n]
    bits = torch.from_numpy(bits.astype(np.float64)).cuda()
    count = bits.sum(1) + before
    assert torch.allclose(lse.double(), count.log()[:, None].expand_as(lse), rtol=0, atol=1e-5)
    want = torch.zeros(n, 128, dtype=torch.float64, device="cuda")
    want[:, :n] = bits / count[:, None]
    assert ((out.double() - want[:, None]).abs() <= want[:, None] * 2.0 ** -7).all()


def test_window_moves_with_depth():
    """The window counts positions in the tree: two drafts of one depth see the same keys before."""
    t = Trees([4], [104], 1, 1, window=10, seed=16, poison=False)
    t.mask.copy_(words_of([0b0001, 0b0010, 0b0101, 0b1101], 1))
    t.q.zero_()
    _, lse = t.run()
    # depths 1, 1, 2, 3 at positions 100, 100, 101, 102: keys before 100 past pos - 10, and the drafts
    assert torch.allclose(lse[:, 0].exp(), torch.tensor([10., 10., 10., 10.], device="cuda"))
    t.window = 2
    _, lse = t.run()
    assert torch.allclose(lse[:, 0].exp(), torch.tensor([2., 2., 2., 3.], device="cuda"))
