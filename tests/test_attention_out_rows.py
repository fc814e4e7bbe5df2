"""The rows of out: layouts in which two of them overlap are refused, any other is
written."""
import pytest
import torch

import prep_token_gb300 as dp
from prep_token_gb300 import _build
from test_cache_abi import _att

D = 128


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return dp.library()


def overlap(T, H, st, sh):
    at = sorted(t * st + h * sh for t in range(T) for h in range(H))
    return any(b - a < D for a, b in zip(at, at[1:]))


LAYOUTS = [(T, H, 8 * a, 8 * b) for T in (2, 3, 5) for H in (2, 4, 6)
           for a in range(16, 120, 5) for b in range(16, 120, 5)]


def test_overlapping_rows_are_refused(lib):
    bad = [x for x in LAYOUTS if overlap(*x)]
    assert len(bad) > 500
    for T, H, st, sh in bad + [(4, 8, 128, 128), (1000, 2, 128, 12800), (2, 1000, 12800, 128),
                               (1 << 20, 1 << 10, 128, 136)]:
        assert _att(lib, T=T, H=H, Hkv=H, ost=st, osh=sh) == 3, (T, H, st, sh)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,st,sh", [x for x in LAYOUTS if not overlap(*x)][::29] + [
    (3, 4, 128, 384), (2, 3, 384, 256)])
def test_any_other_layout_is_written(T, H, st, sh):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from _attn import Batch
    assert not overlap(T, H, st, sh)
    b = Batch([T], [70], H, 2 if H % 2 == 0 else 1, D, seed=T)
    flat = torch.full(((T - 1) * st + (H - 1) * sh + D + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = flat.as_strided((T, H, D), (st, sh, 1))
    got, lse = b.run(out=out)
    b.check(got, lse)
    left = torch.ones_like(flat, dtype=torch.bool)
    left.as_strided((T, H, D), (st, sh, 1)).fill_(False)
    assert (flat[left] == 5).all()
