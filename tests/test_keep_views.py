"""The views of dsa_cache_keep that the host refuses, without a GPU: strides with which
two of a cache's entries would share bytes.  With an empty list nothing is launched."""
import ctypes

import pytest

import prep_token_gb300 as dp
from prep_token_gb300 import _build

A = 0x10000


def _check(shape, pages=8, page=16):
    """The status of a call of no rows on one view."""
    bases, shapes = (ctypes.c_void_p * 1)(A), (ctypes.c_int64 * 5)(*shape)
    return dp.library().dsa_cache_keep(bases, shapes, 1, pages, A, A, 4, 4, A, 3, page, A, A, A, 8, 8, A,
                                       0, 0, A, 0, None, None)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build_library()


@pytest.mark.parametrize("shape", [  # page, token and head stride, heads, bytes
    (4096, 256, 128, 2, 128), (4096, 128, 2048, 2, 128), (256, 2048, 128, 2, 128),
    (8192, 512, 128, 2, 64), (128, 2048, 1024, 2, 128), (4096, 256, 0, 1, 256)])
def test_entries_apart(shape):
    assert _check(shape) == 0


@pytest.mark.parametrize("shape", [
    (4096, 128, 256, 2, 128),    # a token's second head is the token behind the next one
    (4096, 256, 384, 2, 128),    # tokens and heads interleave
    (2048, 256, 128, 2, 128),    # pages of 4096 bytes
    (4080, 256, 128, 2, 128),
    (4096, 128, 1920, 2, 128),   # heads before tokens, one token short
    (128, 1016, 8192, 2, 128),   # pages inside a token's stride, one short
    (128, 128, 8192, 2, 128)])
def test_entries_that_overlap(shape):
    assert _check(shape) == 3


def test_dimensions_of_one():
    """Their strides do not count."""
    assert _check((0, 256, 128, 2, 128), pages=1) == 0
    assert _check((256, 0, 128, 2, 128), page=1) == 0
    assert _check((4096, 256, 0, 1, 256)) == 0
    assert _check((128, 256, 0, 1, 128), pages=4, page=2) == 3
