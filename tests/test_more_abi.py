"""Norm, append, tree attention and cache keep without a GPU: every refusal that
the host makes before any CUDA call, and the binding's checks."""
import ctypes

import pytest
import torch

import prep_token_gb300 as dp
from prep_token_gb300 import _build

A = 0x10000  # fake addresses: only used by calls that must fail validation
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return dp.library()


def _norm(lib, **over):
    a = dict(x=A, xs=64, res=A, rs=64, ro=A, ros=64, gamma=A, eps=1e-6, out=A, os=64, codes=A, cs=64,
             scales=A, ss=2, fmt=0, group=32, T=4, N=64, dtype=0, flags=0, stream=None)
    a.update(over)
    return lib.dsa_rms_norm(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), 3), (dict(T=(1 << 30) + 1), 3), (dict(N=0), 3), (dict(N=60), 3), (dict(N=32776), 3), (dict(dtype=2), 4),
    (dict(flags=2), 4), (dict(flags=8), 4), (dict(eps=0.0), 4), (dict(eps=-1.0), 4),
    (dict(eps=INF), 4), (dict(eps=NAN), 4), (dict(group=64), 4), (dict(group=0), 4),
    (dict(fmt=2), 4), (dict(fmt=-1), 4), (dict(xs=56), 3), (dict(rs=56), 3), (dict(ros=56), 3),
    (dict(os=56), 3), (dict(cs=56), 3), (dict(ss=1), 3), (dict(xs=-64), 3), (dict(xs=1 << 39), 3),
    (dict(x=None), 1), (dict(gamma=None), 1), (dict(out=None, codes=None), 1),
    (dict(scales=None), 1), (dict(res=None), 1), (dict(x=A + 8), 2), (dict(res=A + 2), 2),
    (dict(ro=A + 8), 2), (dict(gamma=A + 4), 2), (dict(out=A + 8), 2), (dict(codes=A + 4), 2),
    (dict(scales=A + 2), 2), (dict(xs=68), 2), (dict(rs=68), 2), (dict(ros=68), 2), (dict(os=68), 2),
    (dict(cs=68), 2), (dict(T=0, x=None, gamma=None), 0)])
def test_norm(lib, over, status):
    assert _norm(lib, **over) == status


def _append(lib, **over):
    a = dict(q=A, qt=4096, qh=128, k=A, kt=4096, kh=128, v=A, vt=4096, vh=128, pos=A, loc=A, cos=A,
             sin=A, cs=32, maxpos=100, qg=None, kg=None, eps=1e-6, qo=A, qot=1024, qoh=128, kc=A,
             vc=A, kp=4096, ktok=256, khead=128, vp=4096, vtok=256, vhead=128, pages=4, ps=16, T=4,
             H=8, Hkv=2, D=128, rope=64, style=0, dtype=0, flags=0, err=None, stream=None)
    a.update(over)
    return lib.dsa_kv_append(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), 3), (dict(H=-1), 3), (dict(Hkv=0), 3), (dict(ps=0), 3), (dict(pages=0), 3),
    (dict(pages=1 << 31), 3), (dict(maxpos=-1), 3), (dict(T=1 << 27, H=8), 3),
    (dict(T=0x7fffffff, H=0x7fffffff), 3), (dict(D=96), 4), (dict(D=256), 4), (dict(dtype=2), 4),
    (dict(rope=-16), 4), (dict(rope=144), 4), (dict(rope=24), 4), (dict(rope=128, D=64), 4),
    (dict(style=2), 4), (dict(flags=4), 4), (dict(qg=A, eps=0.0), 4), (dict(kg=A, eps=NAN), 4),
    (dict(kg=A, eps=INF), 4), (dict(q=None), 1), (dict(qo=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(pos=None), 1), (dict(loc=None), 1), (dict(kc=None), 1),
    (dict(vc=None), 1), (dict(cos=None), 1), (dict(sin=None), 1), (dict(cs=28), 3),
    (dict(qt=0), 3), (dict(kh=0), 3), (dict(vt=-8), 3), (dict(kp=0), 3), (dict(vtok=0), 3),
    (dict(khead=64), 3), (dict(ktok=128), 3), (dict(kp=4000), 3), (dict(vp=1024), 3),
    (dict(qot=512), 3), (dict(qoh=64), 3), (dict(kp=1 << 39), 3), (dict(q=A + 8), 2),
    (dict(k=A + 2), 2), (dict(v=A + 8), 2), (dict(qo=A + 8), 2), (dict(kc=A + 8), 2),
    (dict(vc=A + 8), 2), (dict(pos=A + 4), 2), (dict(loc=A + 4), 2), (dict(cos=A + 8), 2),
    (dict(sin=A + 8), 2), (dict(cs=34), 2), (dict(qg=A + 4), 2), (dict(kg=A + 8), 2),
    (dict(err=A + 2), 2), (dict(qt=4100), 2), (dict(kh=132), 2), (dict(vt=4100), 2),
    (dict(qot=1028), 2), (dict(kp=4100), 2), (dict(vhead=132, vtok=272, vp=8000), 2),
    (dict(T=0, q=None, k=None), 0)])
def test_append(lib, over, status):
    assert _append(lib, **over) == status


def _tree(lib, **over):
    a = dict(q=A, qt=1024, qh=128, k=A, v=A, kp=4096, ktok=256, kh=128, vp=4096, vtok=256, vh=128,
             pages=4, ps=16, bt=A, bts=8, qs=A, lens=A, maxc=100, mask=A, words=2, mstride=2,
             scale=0.1, window=0, sinks=0, out=A, ot=1024, oh=128, lse=A, T=4, B=2, H=8, Hkv=2, D=128,
             dtype=0, flags=0, ws=A, wsb=0, err=None, stream=None)
    a.update(over)
    return lib.dsa_tree_attention(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(mask=None), 1), (dict(mask=A + 2), 2), (dict(words=-1), 3), (dict(mstride=1), 3),
    (dict(mstride=-2), 3), (dict(mstride=1 << 39), 3), (dict(T=-1), 3), (dict(H=7), 3),
    (dict(Hkv=0), 3), (dict(window=-1), 3), (dict(sinks=-1), 3), (dict(bts=6), 3), (dict(D=96), 4),
    (dict(dtype=3), 4), (dict(ps=24), 4), (dict(scale=0.0), 4), (dict(scale=NAN), 4),
    (dict(flags=2), 4), (dict(q=None), 1), (dict(k=None), 1), (dict(bt=None), 1),
    (dict(qs=None), 1), (dict(lens=None), 1), (dict(out=None), 1), (dict(q=A + 8), 2),
    (dict(kp=4100), 2), (dict(ot=64), 3), (dict(lse=A + 2), 2), (dict(maxc=1000, bts=63, wsb=0), 3),
    (dict(maxc=1000, bts=63, ws=None), 1), (dict(maxc=1000, bts=63, ws=A + 8), 2),
    (dict(T=0, q=None), 0), (dict(B=0, q=None), 0)])
def test_tree(lib, over, status):
    assert _tree(lib, **over) == status


def _keep(lib, bases=(A,), shapes=((4096, 256, 128, 2, 128),), n_views=None, pages=8, refs=A, bt=A,
          cols=4, stride=4, lens=A, rows=3, ps=16, which=A, drafted=A, kept=A, ks=8, most=8, nk=A,
          n=2, flags=0, ws=A, wsb=272, err=None, null=False):
    b = (ctypes.c_void_p * max(1, len(bases)))(*bases)
    flat = [x for s in shapes for x in s]
    s = (ctypes.c_int64 * max(1, len(flat)))(*flat)
    return lib.dsa_cache_keep(None if null else b, s, len(bases) if n_views is None else n_views,
                              pages, refs, bt, cols, stride, lens, rows, ps, which, drafted, kept, ks,
                              most, nk, n, flags, ws, wsb, err, None)


@pytest.mark.parametrize("over,status", [
    (dict(n_views=-1), 3), (dict(n_views=257), 3), (dict(pages=0), 3), (dict(pages=1 << 31), 3),
    (dict(ps=0), 3), (dict(null=True), 1), (dict(bases=(0,)), 1),
    (dict(shapes=((4096, 256, 128, 0, 128),)), 3), (dict(shapes=((4096, 256, 128, 2, 0),)), 3),
    (dict(shapes=((4096, 256, 128, 1 << 20, 1 << 20),)), 3), (dict(shapes=((64, 256, 128, 2, 128),)), 3),
    (dict(shapes=((4096, 64, 128, 2, 128),)), 3), (dict(shapes=((4096, 256, 0, 2, 128),)), 3),
    (dict(shapes=((1 << 40, 256, 128, 2, 128),)), 3), (dict(shapes=((4098, 256, 128, 2, 128),)), 2),
    (dict(shapes=((4096, 256, 0, 1, 130),)), 2), (dict(bases=(A + 2,)), 2), (dict(n=-1), 3),
    (dict(n=1025), 3), (dict(most=-1), 3), (dict(ks=7), 3), (dict(rows=-1), 3), (dict(cols=-1), 3),
    (dict(stride=3), 3), (dict(flags=1), 4), (dict(refs=None), 1), (dict(bt=None), 1),
    (dict(lens=None), 1), (dict(which=None), 1), (dict(drafted=None), 1), (dict(kept=None), 1),
    (dict(nk=None), 1), (dict(refs=A + 2), 2), (dict(bt=A + 2), 2), (dict(lens=A + 2), 2),
    (dict(which=A + 1), 2), (dict(drafted=A + 2), 2), (dict(kept=A + 2), 2), (dict(nk=A + 2), 2),
    (dict(err=A + 2), 2), (dict(ws=None), 1), (dict(ws=A + 8), 2), (dict(wsb=271), 3),
    (dict(ks=-1), 3), (dict(ks=0, ws=None), 1), (dict(n=0, refs=None, kept=None), 0)])
def test_keep(lib, over, status):
    assert _keep(lib, **over) == status


def test_binding_refuses_host_tensors(lib):
    x, f = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64)
    i, l = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    kv, cache = torch.zeros(2, 1, 64, dtype=torch.bfloat16), torch.zeros(1, 8, 1, 64, dtype=torch.bfloat16)
    for call in (lambda: dp.dsa_rms_norm(x, f, 1e-6), lambda: dp.dsa_rms_norm_fp8(x, f, 1e-6),
                 lambda: dp.dsa_kv_append(None, kv, kv, l, l, f, f, cache, cache),
                 lambda: dp.dsa_tree_attention(kv, cache, cache, i[None], i, i, 8, i[:, None]),
                 lambda: dp.dsa_cache_keep([cache], i, i[None], i, 8, i, i, i[None], i),
                 lambda: dp.TokenViews([cache])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        dp.dsa_rms_norm(None, f, 1e-6)
