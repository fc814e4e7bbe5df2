"""Windows and sinks of any size that a Python int holds: as large ones as there
are contexts hide, or keep, everything."""
import pytest
import torch

from _attn import Batch
from _pool import Pool
from test_gpu_cache import Device, _cuda  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
HUGE = [2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1, 2 ** 70 + 1]


@pytest.mark.parametrize("n", HUGE)
def test_attention(n):
    b = Batch([3], [200], 4, 1, seed=60)
    whole, z = b.run()
    b.window = n
    out, lse = b.run()
    assert torch.equal(out, whole) and torch.equal(lse, z)
    b.window, b.sinks = 5, n
    out, lse = b.run()
    b.window, b.sinks = 0, 0
    b.check(out, lse)


@pytest.mark.parametrize("n", HUGE)
def test_free(n):
    p = Pool(40, 2, 12, 16, [64])
    p.fill_row(0, 191)
    d = Device(p)
    for q in (p, d):
        q.free([0], window=n)
        q.free([0], window=3, sinks=n)
    assert p.err == 0 and (p.refs > 0).sum() == 12
    d.check(p)


@pytest.mark.parametrize("n", [-1, -2 ** 31, -2 ** 32 + 5, -2 ** 63])
def test_negative_ones_are_refused(n):
    import prep_token_gb300 as dp
    b = Batch([3], [200], 4, 1, seed=61)
    p = Pool(40, 2, 12, 16, [64])
    p.fill_row(0, 191)
    d = Device(p)
    for window, sinks in ((n, 0), (5, n)):
        b.window, b.sinks = window, sinks
        with pytest.raises(dp.DsaError, match="SHAPE"):
            b.run()
        with pytest.raises(dp.DsaError, match="SHAPE"):
            d.free([0], window=window, sinks=sinks)
    d.check(p)
