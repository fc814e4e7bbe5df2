"""dsa_kv_append's kernel for many tokens in every form it is compiled for, and with
every kind of cache and page: that this kernel ran is read off a graph that
captures the call."""
import ctypes
import math

import numpy as np
import pytest
import torch

from test_gpu_append import BF, FP, GPTJ, NEOX, Call, go
from test_gpu_launch_count import rt  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
SMS, STREAM_THREADS = 152, 256  # the direct kernel's CTAs have 128 threads


class KernelNode(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("shared", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def block_of(rt, launch):  # noqa: F811
    """Threads per CTA of the one kernel that launch(stream_handle) captures."""
    cu = ctypes.CDLL("libcuda.so.1")
    torch.cuda.synchronize()
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreateWithFlags(ctypes.byref(stream), 1) == 0
    try:
        assert rt.cudaStreamBeginCapture(stream, 1) == 0
        launch(stream.value)
        assert rt.cudaStreamEndCapture(stream, ctypes.byref(graph)) == 0
        n, node, k = ctypes.c_size_t(1), ctypes.c_void_p(), KernelNode()
        assert rt.cudaGraphGetNodes(graph, ctypes.byref(node), ctypes.byref(n)) == 0
        assert cu.cuGraphKernelNodeGetParams_v2(node, ctypes.byref(k)) == 0
        return k.block[0]
    finally:
        if graph.value:
            rt.cudaGraphDestroy(graph)
        rt.cudaStreamDestroy(stream)


def passes(H, kv, D):
    """Of a token: its rows, 512 / D at a time."""
    at_once = 512 // D
    up = lambda n: -(-n // at_once)  # noqa: E731
    return up(H) + (1 if 2 * kv <= at_once else 2 * up(kv))


def many(H, kv, D, norms, **kw):
    """A call of just as many tokens as the stream kernel is taken from, and a few."""
    T = -(-(40 if norms else 250) * SMS // passes(H, kv, D)) + 5
    return Call(T, H, kv, D, norms=norms, **kw)


def stream_go(rt, c):  # noqa: F811
    go(c)
    out = torch.empty(c.T, *c.q.shape[1:], dtype=c.q.dtype, device="cuda") if c.q is not None else None
    kw = {} if out is None else dict(q_out=out)
    assert block_of(rt, lambda s: c.run(stream=s, **kw)) == STREAM_THREADS


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("style", [NEOX, GPTJ])
@pytest.mark.parametrize("rope", ["none", "least", "whole"])
@pytest.mark.parametrize("norms", [0, 3])
def test_every_form(rt, D, dtype, style, rope, norms):  # noqa: F811
    H, kv = (40, 8) if D == 64 else (18, 3)
    stream_go(rt, many(H, kv, D, norms, dtype=dtype, style=style, page=48,
                       rope={"none": 0, "least": 16, "whole": D}[rope], seed=D + norms))


@pytest.mark.parametrize("layout", ["tokens", "heads", "pairs", "pages"])
@pytest.mark.parametrize("page", [1, 48, 64])
@pytest.mark.parametrize("norms", [0, 2])
def test_pages_and_layouts(rt, layout, page, norms):  # noqa: F811
    stream_go(rt, many(17, 5, 128, norms, layout=layout, page=page, rope=128, style=GPTJ, seed=page))


@pytest.mark.parametrize("H,kv,D", [(0, 24, 64), (0, 9, 128), (8, 2, 128), (16, 2, 64), (1, 12, 128)])
@pytest.mark.parametrize("norms", [0, 1])
def test_rows_of_a_pass(rt, H, kv, D, norms):  # noqa: F811
    """No q, k and v rows in one pass, last passes with one row."""
    stream_go(rt, many(H, kv, D, norms, page=16, rope=D, style=NEOX, dtype=FP, seed=H + kv))


def test_the_threshold(rt):  # noqa: F811
    """One token fewer than the stream kernel is taken from: the direct kernel."""
    for norms, per_sm in ((0, 250), (3, 40)):
        n = passes(8, 2, 128)
        for more, block in ((0, STREAM_THREADS), (-1, 128)):
            c = Call(-(-per_sm * SMS // n) + more, 8, 2, norms=norms)
            q = c.run()
            assert block_of(rt, lambda s: c.run(q_out=q, stream=s)) == block


@pytest.mark.parametrize("D,style", [(64, NEOX), (128, GPTJ)])
@pytest.mark.parametrize("norms", [0, 3])
def test_bad_positions_and_slots(D, style, norms):
    c = many(24, 6, D, norms, page=48, rope=D, style=style, seed=D)
    old = c.k_cache.clone(), c.v_cache.clone()
    good = c.run()
    c.k_cache.copy_(old[0]), c.v_cache.copy_(old[1])
    r = np.random.RandomState(1)
    bad_pos, bad_slot = (torch.from_numpy(r.rand(c.T) < 0.3).cuda() for _ in range(2))
    c.positions[bad_pos] = torch.tensor([-1, 500, 2 ** 50], device="cuda")[
        torch.arange(int(bad_pos.sum()), device="cuda") % 3]
    c.slots[bad_slot] = torch.tensor([-1, c.k_cache.shape[0] * 48, 2 ** 40], device="cuda")[
        torch.arange(int(bad_slot.sum()), device="cuda") % 3]
    out = torch.full_like(good, 9.0)
    c.run(q_out=out)
    assert int(c.err) == 1 | 2
    assert (out[bad_pos] == 9).all() and torch.equal(out[~bad_pos], good[~bad_pos])
    c.q = None
    c.check(None, *old, live=~bad_pos & ~bad_slot)


def test_q_in_place():
    c, d = (many(18, 3, 128, 3, rope=128, style=NEOX, seed=4) for _ in range(2))
    want = d.run()
    assert c.run(q_out=c.q).data_ptr() == c.q.data_ptr()
    assert torch.equal(c.q, want) and not math.isnan(float(want.double().sum()))
