"""Attention over a paged cache on the tensor cores, through the binding,
against the definition in 64 bits (tests/_attn.py derives the tolerance).
Everything in the caches that no query sees is NaN, infinite or huge, and
block-table entries that no query needs name no page."""
import pytest
import torch

from _attn import Batch

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import prep_token_gb300 as dp
    dp.library()


def go(*a, **kw):
    b = Batch(*a, **kw)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = b.run(err_flags=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    b.check(out, lse)
    return b, out, lse


def test_one_token_one_key():
    go([1], [1], 1, 1)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 300])
def test_chunk_of_a_prompt(n, dim, dtype):
    go([n], [n], 8, 2, dim, dtype=dtype, seed=n)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("ctx", [1, 63, 64, 65, 128, 129, 1000, 5000])
def test_single_token(ctx, dim, dtype):
    go([1], [ctx], 16, 2, dim, dtype=dtype, seed=ctx)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 192, 576])
@pytest.mark.parametrize("dim", [64, 128])
def test_page_sizes(page, dim):
    go([70, 1, 5], [333, 410, 5], 4, 2, dim, page=page, seed=page)


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 3), (5, 1), (7, 1), (40, 8), (64, 1), (100, 1),
                                      (128, 1), (256, 2), (12, 4), (130, 2)])
def test_head_layouts(heads, kv):
    go([33, 1], [150, 700], heads, kv, seed=heads)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_mixed_batch(dtype):
    """Chunks, single tokens, an empty sequence, a sequence without new tokens."""
    go([1, 200, 0, 17, 0, 1, 64], [900, 200, 0, 1500, 77, 1, 1000], 16, 4, dtype=dtype, page=16)


def test_more_sequences_than_a_warp_scans_at_once():
    new = [1 + (i * 7) % 5 if i % 9 else 0 for i in range(75)]
    ctx = [n + (i * 131) % 400 for i, n in enumerate(new)]
    go(new, ctx, 8, 1, 64, page=16)


def test_many_sequences_and_kv_heads():
    new = [1 + i % 3 for i in range(160)]
    go(new, [n + (i * 37) % 300 for i, n in enumerate(new)], 32, 16, 64, page=32)


@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 70)])
def test_whole_items(window, sinks):
    """Many tiles over contexts that may pass L2: the CTAs take whole items."""
    import prep_token_gb300 as dp
    assert dp.dsa_paged_attention_workspace_bytes(10000, 3, 16, 16, 64, 200000) == 0
    go([6000, 0, 4000], [6100, 0, 4000], 16, 16, 64, max_context=200000, window=window,
       sinks=sinks, seed=20)


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (64, 0), (100, 4), (128, 128), (129, 300),
                                          (200, 16), (1000, 5), (5000, 3)])
@pytest.mark.parametrize("dim", [64, 128])
def test_window_with_sinks(window, sinks, dim):
    go([200, 1, 1, 30], [700, 1200, 50, 1100], 8, 2, dim, page=16, window=window, sinks=sinks,
       seed=window)


def test_window_of_a_long_context_reads_no_old_page():
    go([1, 4], [40000, 39999], 16, 2, window=300, sinks=4, seed=1)


def test_window_in_many_items():
    go([900, 700], [900, 2500], 16, 16, 64, window=257, sinks=10, seed=2)


def test_rows_that_see_nothing():
    """More new tokens than context: the first ones have no position and see no key."""
    b = Batch([5, 3, 200], [2, 0, 150], 8, 2, seed=3)
    out, lse = b.run()
    assert torch.isneginf(lse[:3]).all() and torch.isneginf(lse[5:8]).all()
    b.check(out, lse)


def test_long_context_single_tokens():
    go([1, 1], [65536, 30001], 16, 2, dtype=FP16, seed=4)


def test_long_chunk():
    go([700], [9000], 16, 2, seed=5)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim,new,kv", [(128, 40, 1), (64, 40, 1), (128, 1, 1), (64, 500, 2)])
def test_peaked_scores_rescale(dim, new, kv, dtype):
    """Scores far above one another, growing along the keys, so that the row's
    reference moves often, in rows of one warp at different blocks and halves.
    Every pass gives the bits of the first, which is checked."""
    b = Batch([new], [4000], 8, kv, dim, dtype=dtype, seed=6, poison=False, q_scale=8.0)
    pages = b.table[0, :63].long()
    b.k[pages] *= torch.linspace(0.05, 4.0, 63 * 64, device="cuda").view(63, 64, 1, 1).to(dtype)
    out, lse = b.run()
    b.check(out, lse)
    for _ in range(10):
        again = b.run()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_equal_scores_average_the_values():
    b = Batch([3], [1000], 4, 1, seed=7, q_scale=0.0)
    out, lse = b.run()
    b.check(out, lse)
    n = torch.tensor([998.0, 999.0, 1000.0], device="cuda")[:, None]
    assert torch.allclose(lse, n.log().expand(3, 4), rtol=1e-6)


def test_padding_rows_are_left_alone():
    b = Batch([3, 150], [10, 200], 4, 1, extra_rows=9, seed=8)
    out = torch.full((162, 4, 128), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((162, 4), 7.0, device="cuda")
    got = b.run(out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    b.check(out, lse)
    assert (out[153:] == 7).all() and (lse[153:] == 7).all()


def test_strides():
    """K and V as slices of one buffer, heads before tokens, q as a slice of a
    fused projection, out inside a wider tensor."""
    b = Batch([40, 1], [300, 500], 8, 2, seed=9)
    pages, P, kv, D = b.k.shape
    both = torch.full((pages, 2, kv, P, D + 8), float("nan"), dtype=BF16, device="cuda")
    both[:, 0, :, :, :D], both[:, 1, :, :, :D] = b.k.permute(0, 2, 1, 3), b.v.permute(0, 2, 1, 3)
    b.k = both[:, 0, :, :, :D].permute(0, 2, 1, 3)
    b.v = both[:, 1, :, :, :D].permute(0, 2, 1, 3)
    wide = torch.full((41, 24, D), float("nan"), dtype=BF16, device="cuda")
    wide[:, 8:16] = b.q
    b.q = wide[:, 8:16]
    table = torch.full((2, b.table.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    table[:, :-5] = b.table
    b.table = table[:, :-5]
    big = torch.full((41, 8, 2 * D), 3.0, dtype=BF16, device="cuda")
    out, lse = b.run(out=big[..., D:])
    b.check(out, lse)
    assert (big[..., :D] == 3).all()


def test_bad_pages_make_their_rows_nan():
    """Only the rows that see the page, and the error bit."""
    b = Batch([100, 1, 1], [400, 900, 100], 4, 1, page=16, seed=10, window=150, sinks=20)
    b.table[0, 330 // 16] = 10 ** 6   # seen by the new tokens from 320 on
    b.table[1, 0] = -3                # a sink
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = b.run(err_flags=err)
    assert int(err.item()) == 2
    b.check(out, lse)
    assert torch.isnan(lse[20:101]).all() and torch.isfinite(lse[:20]).all()
    assert torch.isfinite(lse[101:]).all()


def test_contexts_are_clamped():
    b = Batch([1, 2], [500, 100], 4, 1, seed=11, max_context=130)
    out, lse = b.run()
    b.check(out, lse)


def test_zero_context_capacity():
    b = Batch([2], [0], 4, 1, seed=12)
    out, lse = b.run()
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_default_scale_and_lse_of_the_parts():
    """Two halves of a context joined by their lse give the whole."""
    b = Batch([1], [2048], 8, 1, seed=13, poison=False)
    import prep_token_gb300 as dp
    whole, z = b.run()
    same, _ = dp.dsa_paged_attention(b.q, b.k, b.v, b.table, b.start, b.lens, 2048)
    assert torch.equal(whole, same)
    half = b.lens // 2
    o1, z1 = dp.dsa_paged_attention(b.q, b.k, b.v, b.table, b.start, half, 1024)
    o2, z2 = dp.dsa_paged_attention(b.q, b.k, b.v, b.table[:, 16:].contiguous(), b.start, half, 1024)
    w1, w2 = (z1 - z).exp()[..., None], (z2 - z).exp()[..., None]
    # each half's out is a bf16 value: two half steps of 2^-8 of |out|
    want = o1.double() * w1 + o2.double() * w2
    tol = 3 * 2.0 ** -8 * (o1.double().abs() * w1 + o2.double().abs() * w2 + whole.double().abs())
    assert ((whole.double() - want).abs() <= tol).all()


def test_same_call_same_bits():
    b = Batch([1, 90, 1], [9000, 4000, 20], 16, 2, seed=14)
    out, lse = b.run()
    for _ in range(5):
        again = b.run()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("dim", [64, 128])
def test_keys_from_far_memory_same_bits(dim, window):
    """More keys than L2 holds, each block waited for: every pass gives the bits
    of the first, which is checked."""
    ctx = [3000 + 37 * i for i in range(40)]
    b = Batch([1] * 40, ctx, 32, 8, dim, seed=31, window=window, sinks=5)
    out, lse = b.run()
    b.check(out, lse)
    flush = torch.empty(200_000_000, dtype=torch.uint8, device="cuda")
    for i in range(30):
        flush.fill_(i)
        again = b.run()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1]), f"pass {i}"


def test_graph_and_streams():
    """Captured and replayed on new inputs; two calls at once with a workspace each."""
    import prep_token_gb300 as dp
    b = Batch([1, 40], [3000, 700], 16, 2, seed=15)
    c = Batch([1, 40], [3000, 700], 16, 2, seed=16)
    need = dp.dsa_paged_attention_workspace_bytes(41, 2, 16, 2, 128, 3000)
    assert need > 0
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out, lse = torch.empty_like(b.q), torch.empty((41, 16), device="cuda")
    b.run(out=out, lse=lse, workspace=ws[0])
    b.check(out, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run(out=out, lse=lse, workspace=ws[0])
    b.q.copy_(c.q)
    out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        oc, lc = c.run(workspace=ws[1])
    g.replay()
    torch.cuda.synchronize()
    b.check(out, lse)
    c.check(oc, lc)


def test_explicit_stream_keeps_what_was_allocated_for_it():
    """The call runs late on a stream of its own; what it allocated is not given
    out again to the current stream meanwhile."""
    b = Batch([1, 40], [3000, 700], 16, 2, seed=19)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    out, lse = b.run(stream=side)
    for _ in range(8):  # of the workspace's size, the outputs' size
        torch.full((42_000_000,), 255, dtype=torch.uint8, device="cuda")
        torch.full_like(b.q, 3.0)
    side.synchronize()
    b.check(out, lse)
    again, _ = b.run(stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, again)


def test_pdl_reads_what_the_call_before_it_wrote():
    b = Batch([1, 20], [2000, 300], 8, 1, seed=17)
    for _ in range(4):
        b.q = torch.randn_like(b.q, dtype=torch.float32).to(BF16)
        out, lse = b.run(pdl=True)
        b.q = out
        out, lse = b.run(pdl=True)
        b.check(out, lse)


def test_binding_refusals():
    import prep_token_gb300 as dp
    b = Batch([2], [70], 4, 2, seed=18)

    def call(**over):
        a = dict(q=b.q, k=b.k, v=b.v, table=b.table, start=b.start, lens=b.lens, ctx=70)
        kw = {k: over.pop(k) for k in list(over) if k not in a}
        a.update(over)
        return dp.dsa_paged_attention(a["q"], a["k"], a["v"], a["table"], a["start"], a["lens"],
                                      a["ctx"], **kw)

    for over, what in [
            (dict(q=b.q.half()), "expected"), (dict(q=b.q.float()), "expected"),
            (dict(k=b.k[..., :64]), "differ"), (dict(k=b.k[..., :64], v=b.v[..., :64]), "head_dim"),
            (dict(q=b.q[:, :3]), "multiple"), (dict(table=b.table[:, :1]), "block_table"),
            (dict(table=b.table.long()), "int32"), (dict(lens=b.lens[:0]), "context_lens"),
            (dict(start=b.start[:0]), "query_start"), (dict(ctx=10 ** 6), "block_table"),
            (dict(out=b.q[:1]), "out"), (dict(lse=torch.empty(2, 8, device="cuda")[:, ::2]), "lse"),
            (dict(q=b.q.cpu()), "CUDA")]:
        with pytest.raises((ValueError, TypeError), match=what):
            call(**over)
    for over, what in [
            (dict(scale=0.0), "UNSUPPORTED"), (dict(scale=float("nan")), "UNSUPPORTED"),
            (dict(window=-1), "SHAPE"), (dict(sinks=-1), "SHAPE"),
            (dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), table=b.table.repeat(
                1, 3), ctx=300), "SHAPE")]:
        with pytest.raises(dp.DsaError, match=what):
            call(**over)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim,window", [(128, 0), (64, 0), (128, 100), (64, 100)])
def test_values_that_are_not_finite_touch_only_the_rows_that_see_them(dim, window, dtype):
    """A NaN key, and values that are NaN or infinite, among the new tokens:
    the rows before them (and those whose window has passed them) are as if
    they were not there, the rows that see them are not finite."""
    new, ctx = [300, 1, 40], [420, 300, 700]
    b = Batch(new, ctx, 8, 2, dim, page=32, dtype=dtype, seed=22, window=window,
              sinks=3 if window else 0)
    clean = Batch(new, ctx, 8, 2, dim, page=32, dtype=dtype, seed=22, window=window,
                  sinks=3 if window else 0)
    odd = {200: ("v", float("nan")), 260: ("v", float("inf")), 261: ("v", -float("inf")),
           333: ("k", float("nan")), 419: ("v", float("nan"))}
    for key, (what, x) in odd.items():  # of sequence 0, which has positions 120 .. 419
        page = int(b.table[0, key // 32])
        (b.v if what == "v" else b.k)[page, key % 32, 1, 5] = x
    out, lse = b.run()
    want, z, tol, tol_l = clean.reference()
    heads = torch.arange(8, device="cuda") >= 4  # those of kv head 1
    pos = torch.arange(120, 420, device="cuda")
    hit = torch.zeros(341, dtype=torch.bool, device="cuda")
    for key in odd:
        hit[:300] |= (pos >= key) & (pos < key + window if window else pos >= key)
    hit = hit[:, None] & heads
    assert not torch.isfinite(out).all(-1)[hit].any()
    ok = ~hit
    assert torch.isfinite(out).all(-1)[ok].all() and torch.isfinite(lse)[ok].all()
    assert ((out.double() - want).abs() <= tol)[ok].all()
    assert ((lse.double() - z).abs() <= tol_l)[ok].all()
