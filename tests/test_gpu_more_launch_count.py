"""Launches per call of norm, append, tree attention and cache keep, counted on
graphs that capture one call each."""
import numpy as np
import pytest
import torch

from _tree import Trees
from test_gpu_append import Call
from test_gpu_keep import Pool, random_case
from test_gpu_launch_count import _nodes, rt  # noqa: F401  (a fixture)
from test_gpu_norm import inputs

pytestmark = pytest.mark.gpu


def test_norm(rt):  # noqa: F811
    import prep_token_gb300 as dp
    for T in (1, 5000):
        x, res, gamma = inputs(T, 1024, torch.bfloat16)
        codes, scales, z = dp.dsa_rms_norm_fp8(x, gamma, 1e-6, residual=res)
        assert _nodes(rt, lambda s: dp.dsa_rms_norm_fp8(
            x, gamma, 1e-6, residual=res, codes=codes, scales=scales, residual_out=z, stream=s)) == 1


def test_append(rt):  # noqa: F811
    for T in (3, 6000):
        c = Call(T, 32, 8, norms=3, max_position=8000)
        q = c.run()
        assert _nodes(rt, lambda s: c.run(q_out=q, stream=s)) == 1


@pytest.mark.parametrize("drafts,ctx,count", [([8], [100], 1), ([8, 60], [3000, 90], 2),
                                              ([30] * 64, [300] * 64, 1)])
def test_tree(rt, drafts, ctx, count):  # noqa: F811
    import prep_token_gb300 as dp
    t = Trees(drafts, ctx, 16, 2, poison=False)
    ws = torch.empty(dp.dsa_paged_attention_max_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    out, lse = t.run()
    assert _nodes(rt, lambda s: t.run(out=out, lse=lse, workspace=ws, stream=s)) == count


def test_keep(rt):  # noqa: F811
    import prep_token_gb300 as dp
    p = Pool(*random_case(8, np.random.RandomState(6)))
    d = p.device()
    views = dp.TokenViews(p.views)
    ws = torch.empty(dp.dsa_cache_keep_workspace_bytes(8, p.kept.shape[1]), dtype=torch.uint8,
                     device="cuda")
    assert _nodes(rt, lambda s: dp.dsa_cache_keep(views, *d[:3], p.page, *d[3:], workspace=ws,
                                                  stream=s)) == 2
    none = dp.TokenViews([])
    assert _nodes(rt, lambda s: dp.dsa_cache_keep(none, *d[:3], p.page, *d[3:], workspace=ws,
                                                  stream=s)) == 1
