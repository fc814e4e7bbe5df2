"""The host arrays that the page calls take: bases and page sizes of every cache,
from any iterable of tensors."""
import ctypes

import pytest
import torch

import prep_token_gb300 as dp


@pytest.mark.parametrize("kind", [list, tuple, iter, lambda c: (t for t in c),
                                  lambda c: dict(enumerate(c)).values()])
def test_any_iterable_of_caches(kind):
    caches = [torch.zeros((6, n), dtype=torch.uint8) for n in (4, 132, 64)]
    hold, bases, sizes, n = dp._cache_arrays(kind(caches), 6, torch.device("cpu"))
    assert n == 3 and bases and sizes
    assert list((ctypes.c_uint64 * 3).from_address(bases)) == [t.data_ptr() for t in caches]
    assert list((ctypes.c_int64 * 3).from_address(sizes)) == [4, 132, 64]


@pytest.mark.parametrize("kind", [list, iter])
def test_checks_see_every_cache(kind):
    good, bad = torch.zeros(6, 4), torch.zeros(4, 6).t()
    with pytest.raises(ValueError, match=r"caches\[1\] must be a contiguous"):
        dp._cache_arrays(kind([good, bad]), 6, torch.device("cpu"))
