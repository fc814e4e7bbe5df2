"""Page upkeep without a GPU: every refusal that the host makes before any
CUDA call, and the binding's checks."""
import ctypes

import pytest

import prep_token_gb300 as dp
from prep_token_gb300 import _build

A = 0x10000  # fake addresses: only used by calls that must fail validation


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return dp.library()


def arrays(bases, sizes):
    return (ctypes.c_void_p * max(1, len(bases)))(*bases), \
        (ctypes.c_int64 * max(1, len(sizes)))(*sizes)


def _copy(lib, bases=(A,), sizes=(64,), n_caches=None, pages=8, src=A, dst=A, n=2, flags=0,
          err=None, null=False):
    b, s = arrays(bases, sizes)
    return lib.dsa_cache_copy_pages(None if null else b, s, len(bases) if n_caches is None
                                    else n_caches, pages, src, dst, n, flags, err, None)


CACHES = [(dict(n_caches=-1), 3), (dict(n_caches=129), 3), (dict(pages=0), 3),
          (dict(pages=1 << 31), 3), (dict(null=True), 1), (dict(bases=(A, 0), sizes=(64, 64)), 1),
          (dict(sizes=(0,)), 3), (dict(sizes=(6,)), 2), (dict(sizes=((1 << 30) + 4,)), 3),
          (dict(bases=(A + 2,)), 2), (dict(flags=1), 4), (dict(n=-1), 3), (dict(err=A + 2), 2)]


@pytest.mark.parametrize("over,status", CACHES + [
    (dict(src=None), 1), (dict(dst=None), 1), (dict(src=A + 2), 2), (dict(dst=A + 1), 2),
    (dict(n=0, src=None, dst=None), 0), (dict(bases=(), sizes=()), 0)])
def test_copy_validation(lib, over, status):
    assert _copy(lib, **over) == status


def _fork(lib, bases=(A,), sizes=(64,), n_caches=None, pages=8, refs=A, bt=A, cols=4, stride=4,
          lens=A, rows=3, ps=4, parents=A, children=A, n=2, flags=0, ws=A, wsb=16, err=None,
          null=False):
    b, s = arrays(bases, sizes)
    return lib.dsa_cache_fork(None if null else b, s, len(bases) if n_caches is None else n_caches,
                              pages, refs, bt, cols, stride, lens, rows, ps, parents, children, n,
                              flags, ws, wsb, err, None)


TABLES = [(dict(refs=None), 1), (dict(bt=None), 1), (dict(lens=None), 1), (dict(refs=A + 2), 2),
          (dict(bt=A + 2), 2), (dict(lens=A + 2), 2), (dict(cols=-1), 3), (dict(stride=3), 3),
          (dict(rows=-1), 3), (dict(ps=0), 3)]


@pytest.mark.parametrize("over,status", CACHES + TABLES + [
    (dict(n=1025), 3), (dict(parents=None), 1), (dict(children=None), 1), (dict(ws=None), 1),
    (dict(ws=A + 4), 2), (dict(wsb=15), 3), (dict(parents=A + 2), 2), (dict(children=A + 2), 2),
    (dict(n=0, refs=None, bt=None, lens=None, ws=None, wsb=0), 0)])
def test_fork_validation(lib, over, status):
    assert _fork(lib, **over) == status


def _free(lib, pages=8, refs=A, bt=A, cols=4, stride=4, lens=A, rows=3, ps=4, which=A, n=2,
          window=0, sinks=0, flags=0, err=None):
    return lib.dsa_cache_free(pages, refs, bt, cols, stride, lens, rows, ps, which, n, window,
                              sinks, flags, err, None)


@pytest.mark.parametrize("over,status", TABLES + [
    (dict(pages=0), 3), (dict(pages=1 << 31), 3), (dict(n=-1), 3), (dict(window=-1), 3),
    (dict(sinks=-1), 3), (dict(flags=2), 4), (dict(which=None), 1), (dict(which=A + 2), 2),
    (dict(err=A + 1), 2), (dict(n=0, refs=None, which=None), 0)])
def test_free_validation(lib, over, status):
    assert _free(lib, **over) == status


def _compact(lib, bases=(A,), sizes=(64,), n_caches=None, pages=8, refs=A, bt=A, cols=4, stride=4,
             lens=A, rows=3, ps=4, live=A, flags=0, ws=A, wsb=None, err=None, null=False):
    b, s = arrays(bases, sizes)
    wsb = lib.dsa_cache_compact_workspace_bytes(pages) if wsb is None else wsb
    return lib.dsa_cache_compact(None if null else b, s,
                                 len(bases) if n_caches is None else n_caches, pages, refs, bt,
                                 cols, stride, lens, rows, ps, live, flags, ws, wsb, err, None)


@pytest.mark.parametrize("over,status", [c for c in CACHES if "n" not in c[0]] + TABLES + [
    (dict(pages=(1 << 20) + 1), 3), (dict(live=None), 1), (dict(ws=None), 1), (dict(ws=A + 2), 2),
    (dict(live=A + 2), 2), (dict(wsb=75), 3)])
def test_compact_validation(lib, over, status):
    assert _compact(lib, **over) == status


def test_workspace_sizes(lib):
    assert dp.dsa_cache_fork_workspace_bytes(5) == 40
    assert dp.dsa_cache_fork_workspace_bytes(-1) == 0
    assert dp.dsa_cache_compact_workspace_bytes(8) == 4 * (1 + 2 * 5 + 8)
    assert dp.dsa_cache_compact_workspace_bytes(0) == 0


def test_binding_rejects_cpu_tensors():
    import torch
    i = torch.zeros(4, dtype=torch.int32)
    t = torch.zeros((2, 4), dtype=torch.int32)
    c = [torch.zeros((4, 16), dtype=torch.uint8)]
    for call in (lambda: dp.dsa_cache_copy_pages(c, 4, i, i),
                 lambda: dp.dsa_cache_fork(c, i, t, i, 4, i, i),
                 lambda: dp.dsa_cache_free(i, t, i, 4, i),
                 lambda: dp.dsa_cache_compact(c, i, t, i, 4)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def _att(lib, **over):
    a = dict(q=A, qst=1024, qsh=128, k=A, v=A, ksp=16384, kst=256, ksh=128, vsp=16384, vst=256,
             vsh=128, pages=8, ps=64, bt=A, bts=4, start=A, lens=A, maxc=256, scale=0.1, window=0,
             sinks=0, out=A, ost=1024, osh=128, lse=A, T=4, B=2, H=8, Hkv=2, D=128, dtype=0,
             flags=0, ws=A, wsb=1 << 30, err=None, stream=None)
    a.update(over)
    return lib.dsa_paged_attention(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), 3), (dict(B=-1), 3), (dict(H=0), 3), (dict(Hkv=0), 3), (dict(H=9), 3),
    (dict(maxc=-1), 3), (dict(bts=3), 3), (dict(pages=0), 3), (dict(window=-1), 3),
    (dict(sinks=-1), 3), (dict(D=96), 4), (dict(dtype=2), 4), (dict(H=129, Hkv=1), 4),
    (dict(ps=4), 4), (dict(ps=24), 4), (dict(ps=96), 4), (dict(scale=0.0), 4),
    (dict(scale=-1.0), 4), (dict(scale=float("inf")), 4), (dict(flags=2), 4),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(bt=None), 1),
    (dict(start=None), 1), (dict(lens=None), 1), (dict(out=None), 1), (dict(ws=None), 1),
    (dict(q=A + 8), 2), (dict(k=A + 8), 2), (dict(v=A + 8), 2), (dict(out=A + 8), 2),
    (dict(qst=1028), 2), (dict(ksp=16388), 2), (dict(vsh=124), 2), (dict(osh=132), 2),
    (dict(lse=A + 2), 2), (dict(ws=A + 8), 2), (dict(wsb=1 << 20), 3), (dict(kst=0), 3),
    (dict(ksp=-16384), 3), (dict(T=1 << 29, H=8), 3), (dict(osh=64), 3), (dict(ost=0), 3),
    (dict(T=0, q=None, out=None), 0), (dict(B=0, start=None), 0)])
def test_attention_validation(lib, over, status):
    assert _att(lib, **over) == status


def test_attention_workspace(lib):
    f = lib.dsa_paged_attention_workspace_bytes
    one = f(1, 1, 64, 8, 128, 4096)
    assert one == 304 * 16 + 608 * 128 * (8 + 4 * 128)
    assert f(64, 64, 64, 8, 64, 4096) == 304 * 16 + 608 * 128 * (8 + 4 * 64)
    assert f(1, 1, 64, 8, 128, 128) == 0      # one block: nothing to cut
    assert f(8192, 1, 64, 8, 128, 8192) == one   # keys that L2 holds
    assert f(8192, 1, 64, 8, 128, 65536) == 0    # whole items, one kv head at a time
    assert f(0, 1, 64, 8, 128, 4096) == f(1, 1, 64, 7, 128, 4096) == 0
