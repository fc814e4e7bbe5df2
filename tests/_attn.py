"""Attention over a paged cache in 64 bits, sequence by sequence, from its
definition, and the bound on the kernel's error.

The bound, from the arithmetic, with u the half step of the 16-bit type
(finfo.eps / 2) and A = sum p |v| / sum p:
  * a score: the D products are exact in fp32, their sum and the scaling are
    off by ds = (D + 8) 2^-23 scale sum_d |q_d k_d| (2^-23: the tensor cores'
    adder may truncate), and the exponent's argument c s - c m by 3 roundings
    of numbers up to c max |s|;
  * p: the exponential 2^-21, its rounding to the type u; in fp16 a p 2^-21
    below the largest is subnormal: 2^-25 absolute against a largest p' of at
    least 2^7 (all in units of sum p >= p_max), n of them;
  * sums of n terms in fp32: n 2^-23; the last rounding u |out|.
An error e of every p (relative) moves out by at most 2 e A and lse by e."""
import math

import numpy as np
import torch


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def reference(q, k, v, table, start, lens, scale, window=0, sinks=0):
    """(out, lse, tolerance of out, tolerance of lse) in float64 on q's device;
    rows of no sequence are NaN.  A row that sees a bad page is NaN."""
    T, H, D = q.shape
    pages, P, kv, _ = k.shape
    G, u = H // kv, half_step(q.dtype)
    dev = q.device
    out = torch.full((T, H, D), math.nan, dtype=torch.float64, device=dev)
    lse = torch.full((T, H), math.nan, dtype=torch.float64, device=dev)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    start, lens, table = start.tolist(), lens.tolist(), table.cpu().long()
    for b in range(len(start) - 1):
        n, L = start[b + 1] - start[b], lens[b]
        rows = slice(start[b], start[b + 1])
        if n == 0:
            continue
        pos = torch.arange(L - n, L, device=dev)[:, None]
        key = torch.arange(max(L, 1), device=dev)[None]
        seen = (key <= pos) & (key < L)
        if window:
            seen &= (key > pos - window) | (key < sinks)
        used = seen.any(0).cpu()
        page = table[b][torch.arange(max(L, 1)) // P]
        ok = (page >= 0) & (page < pages)
        bad = (used & ~ok).to(dev)
        take = torch.where(ok & used, page, 0).to(dev)
        slot = (torch.arange(max(L, 1)) % P).to(dev)
        live = (ok & used).to(dev)[:, None]
        for h in range(kv):
            K = torch.where(live, k[take, slot, h].double(), 0)
            V = torch.where(live, v[take, slot, h].double(), 0)
            Q = q[rows, h * G:(h + 1) * G].double()
            s = torch.einsum("tgd,kd->tgk", Q, K) * scale
            mass = torch.einsum("tgd,kd->tgk", Q.abs(), K.abs()) * scale
            hide = ~seen[:, None]
            s = s.masked_fill(hide, -math.inf).masked_fill(bad & ~hide, math.nan)
            z = torch.logsumexp(s, -1)
            p = torch.where(torch.isneginf(z)[..., None], 0, (s - z[..., None]).exp())
            o = torch.einsum("tgk,kd->tgd", p, V)
            A = torch.einsum("tgk,kd->tgd", p, V.abs())
            N = seen.sum(-1).double()[:, None]
            ds = (D + 8) * 2.0 ** -23 * mass.masked_fill(hide, 0).amax(-1) \
                + 4 * 2.0 ** -23 * s.masked_fill(hide, 0).abs().amax(-1)
            e = ds + 2.0 ** -21 + (N + 128) * 2.0 ** -23
            sub = N * (2.0 ** -25 / 2.0 ** 7 if q.dtype == torch.float16 else 2.0 ** -126)
            top = torch.where(seen.any(0)[:, None], V, 0).abs().amax(0)
            at = slice(h * G, (h + 1) * G)
            out[rows, at], lse[rows, at] = o, z
            tol_o[rows, at] = (2 * e + u)[..., None] * A * (1 + u) + u * o.abs() \
                + sub[..., None] * top + 2.0 ** -130
            if q.dtype == torch.float16:
                tol_o[rows, at] += 2.0 ** -25  # out itself may be subnormal
            tol_l[rows, at] = e + 2.0 ** -22 * torch.where(torch.isfinite(z), z, 0).abs()
    return out, lse, tol_o, tol_l


class Batch:
    """Random inputs: lists of new tokens and context lengths, pages of each
    sequence shuffled over a pool; whatever no query sees is poisoned."""

    def __init__(self, new, ctx, heads, kv, dim=128, page=64, dtype=torch.bfloat16, seed=0,
                 window=0, sinks=0, extra_rows=0, extra_pages=2, max_context=None, poison=True,
                 q_scale=2.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = np.random.RandomState(seed)
        B = len(new)
        self.window, self.sinks, self.scale = window, sinks, dim ** -0.5
        self.max_context = max(ctx) if max_context is None else max_context
        cols = max(1, -(-self.max_context // page))
        full, ctx = ctx, [min(c, self.max_context) for c in ctx]
        table = np.full((B, cols), -1, np.int64)
        need = [(b, j) for b in range(B) for j in range(-(-ctx[b] // page))]
        pool = len(need) + extra_pages
        perm = r.permutation(pool)
        seen = np.zeros((pool, page), bool)
        for i, (b, j) in enumerate(need):
            keys = np.arange(j * page, (j + 1) * page)
            first = ctx[b] - new[b]
            low = max(0, first - window + 1) if window else 0
            vis = (keys < ctx[b]) & ((keys >= low) | (keys < sinks)) & (new[b] > 0)
            if vis.any():
                table[b, j] = perm[i]
                seen[perm[i]] = vis
            else:
                table[b, j] = r.choice([-1, pool, 2 ** 31 - 1, -(2 ** 31)])  # never read
        T = sum(new) + extra_rows
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
        self.q = rand(T, heads, dim) * q_scale
        self.k, self.v = rand(pool, page, kv, dim), rand(pool, page, kv, dim)
        if poison:
            dead = torch.from_numpy(~seen).cuda()
            junk = torch.tensor([math.nan, math.inf, -math.inf, 3e4], dtype=dtype, device="cuda")
            self.k[dead] = junk[torch.arange(int(dead.sum()), device="cuda") % 4][:, None, None]
            self.v[dead] = junk[torch.arange(int(dead.sum()), device="cuda") % 3][:, None, None]
        self.table = torch.from_numpy(table).to(torch.int32).cuda()
        self.start = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(full, dtype=torch.int32, device="cuda")

    def run(self, **kw):
        import prep_token_gb300 as dp
        return dp.dsa_paged_attention(self.q, self.k, self.v, self.table, self.start, self.lens,
                                      self.max_context, scale=self.scale, window=self.window,
                                      sinks=self.sinks, **kw)

    def reference(self):
        lens = torch.clamp(self.lens, max=self.max_context)
        return reference(self.q, self.k, self.v, self.table, self.start, lens, self.scale,
                         self.window, self.sinks)

    def check(self, out, lse):
        want, z, tol, tol_l = self.reference()
        T = int(self.start[-1])
        out, lse, want, z = out[:T].double(), lse[:T].double(), want[:T], z[:T]
        nan = torch.isnan(z)
        assert torch.equal(torch.isnan(lse), nan), "NaN rows differ"
        assert torch.equal(torch.isnan(out).all(-1), nan) and torch.equal(torch.isnan(out).any(-1), nan)
        assert torch.equal(torch.isneginf(lse), torch.isneginf(z)), "empty rows differ"
        assert (out[torch.isneginf(z)] == 0).all()
        some = torch.isfinite(z)
        over = ((out - want).abs() / tol[:T])[some]
        over_l = ((lse - z).abs() / tol_l[:T])[some]
        worst = (float(over.max()), float(over_l.max())) if over.numel() else (0.0, 0.0)
        assert worst[0] <= 1 and worst[1] <= 1, f"error / tolerance: out {worst[0]}, lse {worst[1]}"
        return worst
