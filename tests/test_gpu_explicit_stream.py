"""Calls given a stream other than the current one: what they allocate is neither
memory that the current stream still uses nor given out to it too early."""
import pytest
import torch

from _attn import Batch
from _pool import Pool
from test_gpu_cache import Device, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import prep_token_gb300 as dp
    dp.library()


def busy():
    torch.cuda._sleep(40_000_000)  # about 20 ms


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_take_no_memory_that_the_current_stream_still_reads(raw):
    """The only blocks of out's size that are free are some that queued copies read."""
    import prep_token_gb300 as dp
    b = Batch([1, 400], [3000, 700], 64, 8, seed=50)
    want, lse = b.run()
    ws = torch.empty(dp.dsa_paged_attention_max_workspace_bytes(128), dtype=torch.uint8,
                     device="cuda")
    side = torch.cuda.Stream()
    kept = [torch.empty_like(b.q) for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    temps = [torch.full_like(b.q, 3.0) for _ in range(3)]
    torch.cuda.synchronize()
    busy()
    for t, k in zip(temps, kept):
        k.copy_(t)
    del temps, t
    out, _ = b.run(lse=lse, workspace=ws, stream=side.cuda_stream if raw else side)
    side.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    assert all((k == 3.0).all() for k in kept)


def test_outputs_stay_until_the_current_stream_has_read_them():
    b = Batch([1, 40], [3000, 700], 16, 2, seed=51)
    c = Batch([1, 40], [3000, 700], 16, 2, seed=52)
    want, _ = b.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = b.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    busy()
    kept = out.clone()
    del out, lse
    for _ in range(3):  # of the same sizes, on that stream
        c.run(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_page_calls_take_no_workspace_that_the_current_stream_still_writes():
    """Fork and compact: their second kernel reads what the first wrote there."""
    import prep_token_gb300 as dp
    p = Pool(64, 40, 6, 4, [64, 12], seed=1)
    p.fill_row(0, 18)
    p.fill_row(1, 7)
    d = Device(p)
    parents, children = ints([0, 1] * 15), ints(range(2, 32))
    side = torch.cuda.Stream()
    need = max(dp.dsa_cache_fork_workspace_bytes(30), dp.dsa_cache_compact_workspace_bytes(64))
    temps = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (need, need, 240, 512, 1)]
    torch.cuda.synchronize()
    busy()
    for t in temps:
        t.fill_(255)
    del temps, t
    dp.dsa_cache_fork(d.caches, d.refs, d.table, d.lens, 4, parents, children, err_flags=d.err,
                      stream=side)
    live = dp.dsa_cache_compact(d.caches, d.refs, d.table, d.lens, 4, err_flags=d.err, stream=side)
    for _ in range(8):
        torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    p.fork([0, 1] * 15, range(2, 32))
    assert int(live.item()) == p.compact()
    d.check(p)


def test_in_a_capture_that_forks_to_a_side_stream():
    b = Batch([1, 40], [3000, 700], 16, 2, seed=53)
    want, _ = b.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        out, lse = b.run(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        twice = out * 2
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(twice, want * 2)
