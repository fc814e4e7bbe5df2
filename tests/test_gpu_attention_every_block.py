"""Every key block counts once: tests in which a block (or a key) that is lost or
counted twice where work is cut, split and joined moves the results by many
times the tolerance, however long the context.

The values are one-hot by key block, so out holds the weight of every D-th
block.  All terms of its sums are positive, so with u the half step of the
16-bit type each element is off by at most, relative to itself,
  * 2 (ds + 2^-21): the scores' errors ds and the exponential's, in the element
    and in the sum of all weights;
  * u for P's rounding, u for out's own;
  * (N / 16 + 8) 2^-23 for the products' accumulation, 16 keys at a time;
  * dl for the sum of the weights: 18 additions within a half block of 64 keys,
    one per half block and one per part, each 2^-24.
lse is off by ds + 2^-21 + dl and its own last steps (logf's and a sum's, 2^-22
of the numbers added, which with fp16's factor of 2^7 are up to |lse| + 10)."""
import math

import pytest
import torch

from _attn import Batch, half_step

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import prep_token_gb300 as dp
    dp.library()


def check(new, ctx, heads, kv, dim=128, page=64, dtype=BF16, window=0, sinks=0, q_scale=0.0,
          max_context=None, one_key=False):
    b = Batch(new, ctx, heads, kv, dim, page, dtype, seed=sum(ctx), window=window, sinks=sinks,
              q_scale=q_scale, max_context=max_context)
    key = torch.arange(page, device="cuda")
    for s in range(len(new)):
        for j in range(-(-ctx[s] // page)):
            at = int(b.table[s, j])
            if 0 <= at < b.v.shape[0]:
                live = j * page + key < ctx[s]
                hot = torch.nn.functional.one_hot((j * page + key) // 128 % dim, dim).to(dtype)
                b.v[at][live] = hot[live][:, None]
    out, lse = b.run()
    G, u, row = heads // kv, half_step(dtype), 0
    for s, (n, L) in enumerate(zip(new, ctx)):
        if n == 0:
            continue
        pos, keys = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")
        seen = keys <= pos
        if window:
            seen &= (keys > pos - window) | (keys < sinks)
        used = seen.any(0)
        pages = torch.where(used, b.table[s].long()[keys // page], 0)
        group = torch.nn.functional.one_hot(keys // 128, -(-L // 128)).double()
        N = seen.sum(-1).double()[:, None]
        for h in range(kv):
            K = torch.where(used[:, None], b.k[pages, keys % page, h].double(), 0)
            Q = b.q[row:row + n, h * G:(h + 1) * G].double()
            score = torch.einsum("tgd,kd->tgk", Q, K) * b.scale
            z = torch.logsumexp(score.masked_fill(~seen[:, None], -math.inf), -1)
            block = torch.where(seen[:, None], (score - z[..., None]).exp(), 0) @ group
            want = torch.zeros(n, G, dim, dtype=torch.float64, device="cuda")
            want.index_add_(2, torch.arange(group.shape[1], device="cuda") % dim, block)
            mass = torch.einsum("tgd,kd->tgk", Q.abs(), K.abs()).amax(-1) * b.scale
            ds = (dim + 8) * 2.0 ** -23 * mass + 4 * 2.0 ** -23 * score.abs().amax(-1)
            exps = ds + 2.0 ** -21 if q_scale else 0.0  # equal scores: every p is 2^0 or 2^7
            # the parts of a row: at most one per CTA
            dl = (18 + N / 64 + torch.clamp(N / 128 + 1, max=304)) * 2.0 ** -24 if q_scale else 0.0
            tol_l = exps + dl + 2.0 ** -22 * (z.abs() + 10)
            tol = (2 * exps + 2 * u + (N / 16 + 8) * 2.0 ** -23 + dl)[..., None] * want
            if dtype == FP16:
                tol = tol + 2.0 ** -25
            got = out[row:row + n, h * G:(h + 1) * G].double()
            lost = (lse[row:row + n, h * G:(h + 1) * G].double() - z).abs()
            assert (lost <= tol_l).all(), f"lse off by {float((lost / tol_l).max())} tolerances"
            off = (got - want).abs()
            assert (off <= tol).all(), f"out off by {float((off / tol).max())} tolerances"
            # the tests' own reach: a block of which a row sees all keys (a key, where one_key)
            # that is lost moves lse by more than two tolerances, of which errors use one
            whole = (seen[:, None].double() @ group == 128).expand_as(block)
            if whole.any():
                assert float((block / tol_l[..., None])[whole].min()) > 2
            if one_key:
                assert float((1 / N / tol_l).min()) > 2
        row += n


# one token over 38 blocks x 8 kv heads: a block to each of 304 CTAs, one less, one more
BORDERS = [([1], [128 * n + d]) for n in (37, 38, 39, 76) for d in (-1, 0, 1)]
SHAPES = [([1], [65536]), ([1, 1], [65536, 30001]), ([1] * 38, [128 * 5] * 38),
          ([1] * 20, [128 * (3 + i) for i in range(20)]), ([3, 1, 40], [20000, 129, 5000]),
          ([700], [9000]), ([64] * 12, [1000] * 12), ([17, 0, 300], [4000, 0, 6000])]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,ctx", BORDERS)
def test_cuts_at_block_borders(new, ctx, dim, dtype):
    """Equal scores: lse is log N to a fraction of a key."""
    check(new, ctx, 16, 8, dim, dtype=dtype, one_key=True)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,ctx", SHAPES)
def test_equal_scores(new, ctx, dim, dtype):
    check(new, ctx, 16, 2, dim, dtype=dtype, one_key=True)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,ctx", SHAPES)
def test_scores_that_differ(new, ctx, dim, dtype):
    check(new, ctx, 8, 2, dim, page=16, dtype=dtype, q_scale=0.5)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(5000, 300), (1000, 16), (129, 129)])
@pytest.mark.parametrize("new,ctx", [([1, 1], [65536, 30001]), ([700, 1], [9000, 4000])])
def test_windows(new, ctx, window, sinks, dim):
    check(new, ctx, 16, 2, dim, window=window, sinks=sinks, one_key=True)
    check(new, ctx, 16, 2, dim, window=window, sinks=sinks, q_scale=0.5)


@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 130)])
def test_whole_items(window, sinks):
    """A capacity beyond what calls cut: the CTAs take whole items."""
    import prep_token_gb300 as dp
    assert dp.dsa_paged_attention_workspace_bytes(9000, 3, 16, 16, 64, 200000) == 0
    check([5000, 0, 4000], [5100, 0, 4000], 16, 16, 64, max_context=200000, window=window,
          sinks=sinks, one_key=True)
