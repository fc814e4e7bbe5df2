"""Launches per call of paged attention and the pages' upkeep, counted on graphs
that capture one call each."""
import pytest
import torch

from _attn import Batch
from test_gpu_launch_count import _nodes, rt  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,ctx,count", [([1], [100], 1), ([1, 40], [3000, 90], 2),
                                           ([10000], [10000], 1)])
def test_attention(rt, new, ctx, count):  # noqa: F811
    import prep_token_gb300 as dp
    long = new[0] == 10000  # whole items, by the capacity of the table
    b = Batch(new, ctx, 16, 16 if long else 2, 64, poison=False,
              max_context=200000 if long else None)
    T = sum(new)
    need = dp.dsa_paged_attention_workspace_bytes(T, len(new), 16, 16 if long else 2, 64,
                                                  b.max_context)
    assert (need > 0) == (count == 2)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(b.q), torch.empty((T, 16), device="cuda")

    def call(s):
        b.run(out=out, lse=lse, workspace=ws, stream=s)

    call(torch.cuda.current_stream().cuda_stream)
    assert _nodes(rt, call) == count


@pytest.mark.parametrize("tokens,heads", [(8, 32), (64, 8)])  # a tile of 128 rows, or two
def test_whole_items_of_short_contexts(rt, tokens, heads):  # noqa: F811
    """Items enough for the SMs and short: not cut, with a workspace or not used."""
    import prep_token_gb300 as dp
    r = torch.Generator().manual_seed(tokens)
    new = torch.randint(tokens // 2, tokens + 1, (40,), generator=r).tolist()
    ctx = [n + int(torch.randint(0, 400, (1,), generator=r)) for n in new]
    b = Batch(new, ctx, 32, heads, 128, seed=tokens)
    need = dp.dsa_paged_attention_workspace_bytes(sum(new), 40, 32, heads, 128, b.max_context)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(b.q), torch.empty((sum(new), 32), device="cuda")

    def call(s):
        b.run(out=out, lse=lse, workspace=ws, stream=s)

    call(torch.cuda.current_stream().cuda_stream)
    b.check(out, lse)
    assert _nodes(rt, call) == 1


def test_pages(rt):  # noqa: F811
    import prep_token_gb300 as dp
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    caches = [torch.zeros((20, 64), dtype=torch.uint8, device="cuda") for _ in range(3)]
    refs, table, lens = ints(*[0] * 20), torch.full((4, 5), -1, dtype=torch.int32, device="cuda"), ints(0, 0, 0, 0)
    a, b = ints(0, 1), ints(2, 3)
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    live = ints(0)
    calls = [(lambda s: dp.dsa_cache_copy_pages(caches, 20, a, b, stream=s), 1),
             (lambda s: dp.dsa_cache_fork(caches, refs, table, lens, 4, a, b, workspace=ws, stream=s), 2),
             (lambda s: dp.dsa_cache_free(refs, table, lens, 4, b, stream=s), 1),
             (lambda s: dp.dsa_cache_compact(caches, refs, table, lens, 4, live_pages=live,
                                             workspace=ws, stream=s), 2)]
    for call, count in calls:
        call(torch.cuda.current_stream().cuda_stream)
        assert _nodes(rt, call) == count
