"""dsa_kv_append against its definition in 64 bits (the fp32 cos/sin given).

Tolerances, with u the half step of the type: a rotated value is two products,
one rounded before the other's fma: 2^-23 (|a c| + |b s|) more than covers both
roundings.  A norm moves a and b by at most 16 * 2^-24 of themselves: D <= 128
squares, 16 of a lane and 3 shuffles, the mean, eps: (16 + 6) 2^-24, half after
the root, and root, division and the two products."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
EPS = 1e-6
NEOX, GPTJ = 0, 1


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import prep_token_gb300 as dp
    dp.library()


class Call:
    """Random inputs of one call: slices of a fused projection, shuffled slots, a poisoned cache."""

    def __init__(self, T, H, kv, D=128, page=16, rope=64, style=NEOX, dtype=BF, norms=0, seed=0,
                 layout="tokens", max_position=500, extra=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = np.random.RandomState(seed)
        self.T, self.rope, self.style = T, rope, style
        qkv = torch.randn(T, (H + 2 * kv) * D + 8, generator=g, device="cuda").to(dtype) * 2
        self.qkv = qkv
        q, k, v, _ = qkv.split([H * D, kv * D, kv * D, 8], 1)
        self.q = q.unflatten(1, (H, D)) if H else None
        self.k, self.v = k.unflatten(1, (kv, D)), v.unflatten(1, (kv, D))
        pages = -(-T // page) + extra
        shape = {"tokens": (2, pages, page, kv, D), "heads": (2, pages, kv, page, D),
                 "pairs": (pages, page, kv, 2, D), "pages": (pages, 2, page, kv, D)}[layout]
        whole = torch.full(shape, math.nan, device="cuda", dtype=dtype)
        both = {"tokens": lambda w: w, "heads": lambda w: w.transpose(2, 3),
                "pairs": lambda w: w.permute(3, 0, 1, 2, 4), "pages": lambda w: w.transpose(0, 1)}
        self.whole, (self.k_cache, self.v_cache) = whole, both[layout](whole)
        up = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.slots = up(r.permutation(pages * page)[:T].astype(np.int64))
        self.positions = up(r.randint(0, max_position, T).astype(np.int64))
        angle = torch.rand(max_position, max(rope // 2, 4) + 4, generator=g, device="cuda",
                           dtype=torch.float64) * 7
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        gamma = torch.rand(2, D, generator=g, device="cuda") * 2 - 0.5
        self.q_gamma = gamma[0] if norms & 1 else None
        self.k_gamma = gamma[1] if norms & 2 else None
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, **kw):
        import prep_token_gb300 as dp
        return dp.dsa_kv_append(
            self.q, self.k, self.v, self.positions, self.slots, self.cos, self.sin, self.k_cache,
            self.v_cache, rope_dim=self.rope, rope_style=self.style, q_gamma=self.q_gamma,
            k_gamma=self.k_gamma, eps=EPS, err_flags=self.err, **kw)

    def rows(self, x, gamma):
        """(rows in 64 bits, tolerance)"""
        y, rel = x.double(), 2.0 ** -23
        if gamma is not None:
            y = y / (y.square().mean(-1, keepdim=True) + EPS).sqrt() * gamma.double()
            rel += 16 * 2.0 ** -24
        r, h = self.rope, self.rope // 2
        pos = self.positions.clamp(0, self.cos.shape[0] - 1)
        c, s = (t[pos, :h].double()[:, None] for t in (self.cos, self.sin))
        a, b = (slice(0, h), slice(h, r)) if self.style == NEOX else (slice(0, r, 2), slice(1, r, 2))
        out, mass = y.clone(), y.abs()
        if r:
            ya, yb = y[..., a], y[..., b]
            out[..., a], out[..., b] = ya * c - yb * s, yb * c + ya * s
            mass[..., a] = (ya * c).abs() + (yb * s).abs()
            mass[..., b] = (yb * c).abs() + (ya * s).abs()
        u = torch.finfo(x.dtype).eps / 2
        tiny = 2.0 ** -25 if x.dtype == FP else 2.0 ** -134
        return out, out.abs() * u * (1 + 2.0 ** -18) + mass * rel * (1 + u) + tiny

    def check(self, q_out, k0, v0, live=None):
        """live: tokens whose K and V are written; k0, v0: the caches before the call."""
        live = torch.ones(self.T, dtype=torch.bool, device="cuda") if live is None else live
        if self.q is not None:
            want, tol = self.rows(self.q, self.q_gamma)
            assert ((q_out.double() - want).abs() <= tol).all()
        P = self.k_cache.shape[1]
        slots = self.slots[live]
        want, tol = self.rows(self.k, self.k_gamma)
        got = self.k_cache[slots // P, slots % P].double()
        assert ((got - want[live]).abs() <= tol[live]).all()
        v0[slots // P, slots % P] = self.v[live]
        k0[slots // P, slots % P] = self.k_cache[slots // P, slots % P]
        for new, old in ((self.k_cache, k0), (self.v_cache, v0)):
            assert torch.equal(new.contiguous().view(torch.int16), old.contiguous().view(torch.int16))


def go(c, **kw):
    old = c.k_cache.clone(), c.v_cache.clone()
    c.check(c.run(**kw), *old)
    assert int(c.err) == 0


@pytest.mark.parametrize("T", [1, 2, 33, 700])
@pytest.mark.parametrize("H,kv,D", [(64, 8, 128), (5, 1, 128), (1, 1, 64), (24, 24, 64), (16, 2, 64),
                                    (0, 3, 128), (7, 7, 128)])
@pytest.mark.parametrize("norms", [0, 3])
def test_heads(T, H, kv, D, norms):
    go(Call(T, H, kv, D, dtype=BF if T % 2 else FP, norms=norms, seed=T + H))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("style", [NEOX, GPTJ])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_rope_dims(D, style, dtype):
    for rope in range(0, D + 1, 16):
        for norms in range(4):
            go(Call(13, 6, 2, D, rope=rope, style=style, dtype=dtype, norms=norms, seed=rope + norms))


@pytest.mark.parametrize("page", [1, 3, 16, 48, 64, 256])
@pytest.mark.parametrize("layout", ["tokens", "heads", "pairs", "pages"])
def test_pages_and_layouts(page, layout):
    go(Call(150, 8, 4, 128, page=page, layout=layout, seed=page))


@pytest.mark.parametrize("H,kv,D", [(8, 2, 128), (32, 8, 128), (4, 1, 128), (16, 2, 64), (9, 5, 64),
                                    (0, 1, 128), (0, 24, 128), (1, 1, 64), (64, 1, 128)])
@pytest.mark.parametrize("norms", [0, 1, 2, 3])
def test_many_tokens(H, kv, D, norms):
    go(Call(9000, H, kv, D, page=64, rope=D // 2, style=kv % 2, norms=norms, max_position=9000,
            dtype=FP if norms == 1 else BF))


def test_bad_positions_and_slots_of_many():
    c = Call(9000, 8, 2, norms=2, seed=5)
    old = c.k_cache.clone(), c.v_cache.clone()
    good = c.run()
    c.k_cache.copy_(old[0]), c.v_cache.copy_(old[1])
    r = np.random.RandomState(1)
    bad_pos = torch.from_numpy(r.rand(9000) < 0.1).cuda()
    bad_slot = torch.from_numpy(r.rand(9000) < 0.1).cuda()
    c.positions[bad_pos] = torch.tensor([-1, 500, 2 ** 50], device="cuda")[
        torch.arange(int(bad_pos.sum()), device="cuda") % 3]
    c.slots[bad_slot] = torch.tensor([-1, 2 ** 40], device="cuda")[
        torch.arange(int(bad_slot.sum()), device="cuda") % 2]
    out = torch.full_like(good, 9.0)
    c.run(q_out=out)
    assert int(c.err) == 1 | 2
    assert (out[bad_pos] == 9).all() and torch.equal(out[~bad_pos], good[~bad_pos])
    c.q = None
    c.check(None, *old, live=~bad_pos & ~bad_slot)


def test_q_in_place_and_given():
    c = Call(40, 8, 2, seed=3)
    want = c.run()
    c.k_cache.fill_(math.nan)
    out = torch.full((50, 8, 128), math.nan, dtype=BF, device="cuda")
    assert c.run(q_out=out).data_ptr() == out.data_ptr()
    assert torch.equal(out[:40], want) and torch.isnan(out[40:]).all()
    got = c.run(q_out=c.q)
    assert torch.equal(got, want) and torch.equal(c.q, want)
    turned = torch.empty(8, 40, 128, dtype=BF, device="cuda").transpose(0, 1)  # heads before tokens
    c = Call(40, 8, 2, seed=3)
    assert torch.equal(c.run(q_out=turned), want)


def test_fewer_tokens_than_rows():
    c = Call(30, 4, 2, seed=4)
    old = c.k_cache.clone(), c.v_cache.clone()
    q = c.run(num_tokens=11)
    assert q.shape[0] == 11
    c.T, c.q, c.k, c.v = 11, c.q[:11], c.k[:11], c.v[:11]
    c.positions, c.slots = c.positions[:11], c.slots[:11]
    c.check(q, *old)


def test_bad_positions_and_slots():
    c = Call(12, 4, 2, seed=5)
    old = c.k_cache.clone(), c.v_cache.clone()
    good = c.run()
    c.k_cache.copy_(old[0]), c.v_cache.copy_(old[1])
    n = c.k_cache.shape[0] * c.k_cache.shape[1]
    c.positions[[2, 7]] = torch.tensor([-1, 500], device="cuda")
    c.slots[[3, 8, 9]] = torch.tensor([-1, n, 2 ** 40], device="cuda")
    out = torch.full_like(good, 9.0)
    c.run(q_out=out)
    assert int(c.err) == 1 | 2
    bad_pos = torch.zeros(12, dtype=torch.bool, device="cuda")
    bad_pos[[2, 7]] = True
    assert (out[bad_pos] == 9).all() and torch.equal(out[~bad_pos], good[~bad_pos])
    live = ~bad_pos
    live[[3, 8, 9]] = False
    c.q = None
    c.check(None, *old, live=live)


def test_nan_stays_in_its_head():
    c = Call(6, 4, 2, norms=3, seed=6)
    c.q[2, 1, 100] = math.nan
    c.k[3, 0, 5] = math.inf
    got = c.run()
    bad = torch.isnan(got).any(-1)
    assert bad[2, 1] and int(bad.sum()) == 1
    P = c.k_cache.shape[1]
    k = c.k_cache[c.slots // P, c.slots % P]
    assert torch.isnan(k[3, 0]).any() and int(torch.isnan(k).any(-1).sum()) == 1


def test_captured_with_the_table_replaced():
    c = Call(64, 16, 2, seed=7)
    import prep_token_gb300 as dp
    out = torch.empty(64, 16, 128, dtype=BF, device="cuda")
    c.run(q_out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(q_out=out, pdl=True)
        c.run(q_out=out, pdl=True)
    d = Call(64, 16, 2, seed=8)
    for name in ("qkv", "positions", "slots", "cos", "sin"):
        getattr(c, name).copy_(getattr(d, name))
    c.whole.fill_(math.nan)
    old = c.k_cache.clone(), c.v_cache.clone()
    graph.replay()
    c.check(out, *old)
    call = dp.prepare_kv_append(c.q, c.k, c.v, c.positions, c.slots, c.cos, c.sin, c.k_cache,
                                c.v_cache, q_out=out, err_flags=c.err)
    out.zero_()
    assert call() is out
    c.check(out, *old)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=side)
    side.synchronize()
    assert torch.equal(got, out) and int(c.err) == 0


def test_empty():
    c = Call(0, 4, 2)
    assert c.run().shape == (0, 4, 128)
