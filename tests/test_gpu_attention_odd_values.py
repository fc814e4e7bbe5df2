"""Keys and values that are not finite, where rows see them: lse is the log of
the sum over the scores whatever the values hold, a key whose score is -inf has
weight 0, one whose score is NaN or +inf makes its rows NaN -- in blocks that
every row sees whole as in those at an edge, cut between CTAs or not, with one
query tile or two."""
import pytest
import torch

from _attn import Batch, reference

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import prep_token_gb300 as dp
    dp.library()


# (new tokens, context) of each sequence: single tokens that are cut between
# many CTAs; chunks of two tiles; whole items of short contexts, in one tile and two
SHAPES = {"one token, cut": [(1, 4000)], "single tokens": [(1, 900), (1, 300), (1, 1500)],
          "chunk": [(300, 700)], "long chunk": [(500, 3000)],
          "short, one tile": [(5, 200 + i) for i in range(60)],
          "short, two tiles": [(60, 260 + i) for i in range(60)]}


def pair(shape, dim, dtype, seed=40, **kw):
    """The same batch twice: one to put odd values into, one left clean."""
    new, ctx = zip(*SHAPES[shape])
    return [Batch(list(new), list(ctx), 16, 2, dim, page=32, dtype=dtype, seed=seed, **kw)
            for _ in range(2)]


def put(b, cache, seq, key, dim, x, head=1):
    cache[int(b.table[seq, key // 32]), key % 32, head, dim] = x


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("shape", SHAPES)
def test_lse_does_not_depend_on_the_values(shape, window, dim, dtype):
    """In sequence 0 a NaN and infinities among the values: far from the new
    tokens, next to them, at a window's edge, and in the last key."""
    b, clean = pair(shape, dim, dtype, window=window, sinks=3 if window else 0)
    n, L = SHAPES[shape][0]
    odd = {1: NAN, 70: INF, L - n - 20: -INF, max(0, L - n - 149): NAN, L - n: INF, L - 1: NAN}
    for i, (key, x) in enumerate(odd.items()):
        if int(b.table[0, key // 32]) in range(b.k.shape[0]):
            put(b, b.v, 0, key, 7 * i, x)
    out, lse = b.run()
    want, z, tol, tol_l = clean.reference()
    assert torch.isfinite(lse).all()
    assert ((lse.double() - z).abs() <= tol_l).all()
    heads = torch.arange(16, device="cuda") >= 8  # those of kv head 1
    pos = torch.arange(L - n, L, device="cuda")
    ok = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    for i, key in enumerate(odd):
        sees = pos >= key
        if window:
            sees &= (key > pos - window) | (key < 3)
        hit = torch.zeros_like(ok)
        hit[:n] = sees[:, None] & heads
        assert not torch.isfinite(out[..., 7 * i][hit]).any(), f"key {key}"
        ok &= ~hit
    assert ((out.double() - want).abs() <= tol)[ok].all()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("key", [0, 130, -1])  # the first, an inner one, the last before the new
@pytest.mark.parametrize("shape", SHAPES)
def test_a_score_of_minus_infinity_has_weight_zero(shape, key, dim, dtype):
    """As if the key were not in the context."""
    new, ctx = zip(*SHAPES[shape])
    b, _ = pair(shape, dim, dtype, seed=41)
    n, L = SHAPES[shape][0]
    key = L - n - 1 if key < 0 else key
    b.q[:n, :, 9] = b.q[:n, :, 9].abs() + 0.5
    put(b, b.k, 0, key, 9, -INF, slice(None))
    out, lse = b.run()
    k, v = (c[b.table[0, :-(-L // 32)].long()].flatten(0, 1)[:L] for c in (b.k, b.v))
    keep = torch.arange(L, device="cuda") != key
    one = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    want, z, tol, tol_l = reference(b.q[:n], k[keep][None], v[keep][None], one(0)[:, None],
                                    one(0, n), one(L - 1), b.scale)
    assert ((out[:n].double() - want).abs() <= tol).all()
    assert ((lse[:n].double() - z).abs() <= tol_l).all()


@pytest.mark.parametrize("x", [NAN, INF])
@pytest.mark.parametrize("key", [0, 130, -1])
@pytest.mark.parametrize("shape", SHAPES)
def test_a_score_of_nan_or_infinity_makes_the_row_nan(shape, key, x):
    b, clean = pair(shape, 128, BF16, seed=42)
    n, L = SHAPES[shape][0]
    key = L - n - 1 if key < 0 else key
    b.q[:n, :, 9] = clean.q[:n, :, 9] = b.q[:n, :, 9].abs() + 0.5
    put(b, b.k, 0, key, 9, x)
    out, lse = b.run()
    want, z, tol, tol_l = clean.reference()
    hit = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    hit[:n, 8:] = True
    assert torch.isnan(lse[hit]).all() and torch.isnan(out[hit]).all()
    assert ((out.double() - want).abs() <= tol)[~hit].all()
    assert ((lse.double() - z).abs() <= tol_l)[~hit].all()


def test_rows_all_of_whose_scores_are_minus_infinity():
    b, _ = pair("one token, cut", 64, BF16, seed=43)
    b.q[..., 9] = 1
    b.k[..., 9] = -INF
    b.k[..., :9] = 0
    b.k[..., 10:] = 0
    out, lse = b.run()
    assert (out == 0).all() and torch.isneginf(lse).all()
