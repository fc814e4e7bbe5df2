"""Calls in their usual form are marshalled in C++, all others through ctypes: both
give the same, and what is out of the ordinary finds its way."""
import pytest
import torch

from _tree import Trees
from test_gpu_append import Call
from test_gpu_keep import Pool, random_case
from test_gpu_norm import inputs

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import prep_token_gb300 as dp
    dp.library()


class Ways:
    """Counts how often the marshalling in C++ carries a call out."""

    def __init__(self, monkeypatch):
        import prep_token_gb300 as dp
        self.real, self.done, self.left = dp._marshal(), 0, 0
        monkeypatch.setattr(dp, "_marshal", lambda: self)

    def __getattr__(self, name):
        f = getattr(self.real, name)

        def call(*args):
            got = f(*args)
            if got is NotImplemented:
                self.left += 1
            else:
                self.done += 1
            return got
        return call


@pytest.fixture
def ways(monkeypatch):
    return Ways(monkeypatch)


def same(a, b):
    a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and x.shape == y.shape and x.device == y.device
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm(ways, residual, dtype):
    import prep_token_gb300 as dp
    x, res, gamma = inputs(37, 1032, dtype)
    res = res if residual else None
    side = torch.cuda.current_stream()
    for group in (32, 128):
        for s in (torch.float32, torch.float8_e8m0fnu):
            same(dp.dsa_rms_norm_fp8(x, gamma, 1e-5, residual=res, group=group, scale_dtype=s),
                 dp.dsa_rms_norm_fp8(x, gamma, 1e-5, residual=res, group=group, scale_dtype=s,
                                     stream=side))
    same(dp.dsa_rms_norm(x[:, 8:1032], gamma[8:], 1e-5, residual=None if res is None else res[:, 8:]),
         dp.dsa_rms_norm(x[:, 8:1032], gamma[8:], 1e-5, residual=None if res is None else res[:, 8:],
                         stream=side))
    assert (ways.done, ways.left) == (5, 0)


def test_append(ways):
    for kw in (dict(norms=3), dict(rope=0), dict(style=1, dtype=FP, D=64), dict(H=0), dict(layout="heads")):
        kw = dict(dict(T=21, H=8, kv=2), **kw)
        c, d = Call(seed=1, **kw), Call(seed=1, **kw)
        a, b = c.run(), d.run(stream=torch.cuda.current_stream())
        if kw["H"]:
            same(a, b)
        same(c.whole, d.whole)
    assert (ways.done, ways.left) == (5, 0)


def test_tree(ways):
    for kw in (dict(), dict(window=50, sinks=3), dict(dtype=FP, dim=64), dict(poison=False)):
        t = Trees([20, 1, 64], [300, 2000, 90], 16, 2, masks="any", seed=2, **kw)
        same(t.run(), t.run(stream=torch.cuda.current_stream()))
        t.scale = None
        same(t.run(pdl=True), t.run(stream=torch.cuda.current_stream()))
    t.window = 2 ** 40
    same(t.run(), t.run(stream=torch.cuda.current_stream()))
    assert (ways.done, ways.left) == (9, 0)


def test_keep(ways):
    import numpy as np
    p = Pool(*random_case(9, np.random.RandomState(1)), shapes=((4, 64), (8,)))
    assert p.check() == 0
    assert (ways.done, ways.left) == (1, 0)


def test_out_of_the_ordinary(ways):
    """Left to the way through ctypes, which refuses as it does, or carries the call out."""
    import prep_token_gb300 as dp
    x, res, gamma = inputs(5, 256, BF)
    for bad, error in ((dict(x=x.float()), TypeError), (dict(x=x.cpu()), ValueError),
                       (dict(x=x.t()), ValueError), (dict(x=x[0]), ValueError),
                       (dict(gamma=gamma[:100]), ValueError), (dict(gamma=gamma.half()), TypeError),
                       (dict(residual=res[:3]), ValueError), (dict(residual=res.half()), TypeError),
                       (dict(x=None), TypeError), (dict(group=64), ValueError),
                       (dict(group=0), ValueError)):
        kw = dict(dict(x=x, gamma=gamma, eps=1e-6), **bad)
        with pytest.raises(error):
            dp.dsa_rms_norm_fp8(kw.pop("x"), kw.pop("gamma"), kw.pop("eps"), **kw)
    assert ways.done == 0
    with pytest.raises(dp.DsaError, match="UNSUPPORTED"):
        dp.dsa_rms_norm(x, gamma, -1.0)
    with pytest.raises(dp.DsaError, match="ALIGN"):
        dp.dsa_rms_norm(x[:, 1:249], gamma[:248].clone(), 1e-6)
    assert ways.done == 2
    got = dp.dsa_rms_norm_fp8(x, gamma, 1e-6, scale_dtype=torch.uint8)
    same(got[1], dp.dsa_rms_norm_fp8(x, gamma, 1e-6, scale_dtype=torch.float8_e8m0fnu)[1].view(torch.uint8))
    t = Trees([4], [40], 8, 2)
    for change in (lambda: t.lens.long(), lambda: t.lens.cpu()):
        with pytest.raises((TypeError, ValueError)):
            dp.dsa_tree_attention(t.q, t.k, t.v, t.table, t.start, change(), 40, t.mask)
    with pytest.raises(ValueError):
        dp.dsa_tree_attention(t.q, t.k, t.v, t.table, t.start, t.lens, 400, t.mask)
    with pytest.raises(ValueError):
        dp.dsa_tree_attention(t.q, t.k, t.v, t.table, t.start, t.lens, 40, t.mask[:3])
    with pytest.raises(dp.DsaError, match="SHAPE"):
        dp.dsa_tree_attention(t.q, t.k, t.v, t.table, t.start, t.lens, 40, t.mask, window=-1)
    c = Call(4, 4, 2)
    c.slots = c.slots[:3]
    with pytest.raises(ValueError):
        c.run()
    c = Call(4, 4, 2, rope=64)
    c.rope = 24
    with pytest.raises(dp.DsaError, match="UNSUPPORTED"):
        c.run()
    c.rope = 4096  # more than the table holds
    with pytest.raises(ValueError):
        c.run()


def test_on_the_current_stream_and_in_a_graph():
    import prep_token_gb300 as dp
    x, res, gamma = inputs(300, 2048, BF, 4)
    want = dp.dsa_rms_norm_fp8(x, gamma, 1e-6, residual=res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = dp.dsa_rms_norm_fp8(x, gamma, 1e-6, residual=res)
    side.synchronize()
    same(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dp.dsa_rms_norm_fp8(x, gamma, 1e-6, residual=res)
    for t in got:
        t.view(torch.uint8).zero_()
    graph.replay()
    same(got, want)


def test_threads():
    """Calls of several Python threads at once, each on a stream of its own."""
    import threading

    import prep_token_gb300 as dp
    sets = [inputs(64 + i, 1024, BF, 10 + i) for i in range(4)]
    want = [dp.dsa_rms_norm_fp8(x, gamma, 1e-6, residual=res) for x, res, gamma in sets]
    torch.cuda.synchronize()
    got = [None] * len(sets)

    def work(i):
        x, res, gamma = sets[i]
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got[i] = [dp.dsa_rms_norm_fp8(x, gamma, 1e-6, residual=res) for _ in range(100)]
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
        assert not t.is_alive()
    for w, results in zip(want, got):
        assert len(results) == 100
        for g in results:
            same(g, w)
