"""What is not finite in dsa_kv_append: an infinity under a norm makes its own place,
and the one that it turns with, NaN, and the others of its head 0, as the definition
in 64 bits has it."""
import math

import pytest
import torch

from test_gpu_append import BF, FP, GPTJ, NEOX, Call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import prep_token_gb300 as dp
    dp.library()


def spoil(x, values):
    """One of the values at a place of its own in each (token, head) row, every place in turn."""
    T, heads, D = x.shape
    n = torch.arange(T * heads, device="cuda")
    flat = x.reshape(T * heads, D).clone()
    flat[n, n % D] = torch.tensor(values, dtype=x.dtype, device="cuda")[(n // D) % len(values)]
    x.copy_(flat.view(T, heads, D))


@pytest.mark.parametrize("T", [130, 4000])  # both kernels
@pytest.mark.parametrize("style", [NEOX, GPTJ])
@pytest.mark.parametrize("D,rope", [(64, 16), (64, 48), (64, 64), (128, 0), (128, 16), (128, 64), (128, 112)])
@pytest.mark.parametrize("norms", [0, 1, 3])
def test_infinities(T, style, D, rope, norms):
    for dtype in (BF, FP):
        c = Call(T, 9, 3, D, rope=rope, style=style, norms=norms, dtype=dtype, seed=rope)
        for x in (c.q, c.k, c.v):
            spoil(x, [math.inf, -math.inf])
        got = c.run()
        P = c.k_cache.shape[1]
        k, v = (t[c.slots // P, c.slots % P] for t in (c.k_cache, c.v_cache))
        for out, x, gamma in ((got, c.q, c.q_gamma), (k, c.k, c.k_gamma)):
            want, _ = c.rows(x, gamma)
            if gamma is not None:
                assert torch.equal(torch.isnan(out), torch.isnan(want))
                assert (out[~torch.isnan(out)] == 0).all()
            else:  # rows as they were but for the pair that turns
                assert torch.equal(torch.isfinite(out), torch.isfinite(want))
        assert torch.equal(v, c.v)
