"""The workspace of paged attention: one of the stated largest size serves every
call, whatever the order of their sizes."""
import itertools

import pytest
import torch

import prep_token_gb300 as dp
from prep_token_gb300 import _build
from test_cache_abi import _att


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return dp.library()


@pytest.mark.parametrize("D", [64, 128])
def test_the_largest_size_serves_every_call(lib, D):
    most = dp.dsa_paged_attention_max_workspace_bytes(D)
    sizes = [dp.dsa_paged_attention_workspace_bytes(T, B, kv * G, kv, D, ctx)
             for T, B, kv, G, ctx in itertools.product(
                 [1, 2, 64, 1000, 8192, 10 ** 6], [1, 2, 64, 5000], [1, 8, 16, 500], [1, 8, 128],
                 [1, 128, 129, 5000, 65536, 10 ** 6, 1 << 30])]
    assert max(sizes) == most and set(sizes) == {0, most}
    assert dp.dsa_paged_attention_max_workspace_bytes(0) == 0


def test_a_prompt_needs_none_and_its_decode_step_does(lib):
    """The size is not monotone, and a byte less than the call's is refused."""
    assert dp.dsa_paged_attention_workspace_bytes(8192, 1, 64, 8, 128, 65536) == 0
    need = dp.dsa_paged_attention_workspace_bytes(1, 1, 64, 8, 128, 65536)
    assert need == dp.dsa_paged_attention_max_workspace_bytes(128)
    big = dict(T=1, B=1, H=64, Hkv=8, maxc=65536, bts=1024)
    assert _att(lib, wsb=need - 1, **big) == 3


@pytest.mark.parametrize("T,B,H,kv,ctx", [(116000, 1, 1, 1, 1 << 30), (116000, 1, 1, 1, 400_000_000),
                                          (900, 1, 128, 1, 400_000_000),
                                          (4_000_000, 70_000, 1, 1, 10_000_000)])
def test_no_cut_where_a_head_has_more_key_blocks_than_32_bits_count(lib, T, B, H, kv, ctx):
    """The place of a cut in a sequence is a 32-bit number of key blocks."""
    tiles, blocks = -(-T // (128 // (H // kv))), -(-ctx // 128)
    assert tiles * blocks >= 1 << 31
    assert dp.dsa_paged_attention_workspace_bytes(T, B, H, kv, 64, ctx) == 0
    # half the rows, and few enough keys: cut as before
    assert dp.dsa_paged_attention_workspace_bytes(T // 2, B, H, kv, 64, ctx // 16) > 0


@pytest.mark.gpu
def test_one_workspace_for_a_prompt_and_its_decode_steps():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from _attn import Batch
    ws = torch.empty(dp.dsa_paged_attention_max_workspace_bytes(64), dtype=torch.uint8,
                     device="cuda")
    for new, ctx in (([9000], [9000]), ([1], [9001]), ([1, 40], [9002, 100]), ([4000], [5000])):
        b = Batch(new, ctx, 16, 16, 64, max_context=200000, seed=sum(new))
        out, lse = b.run(workspace=ws)
        b.check(out, lse)
