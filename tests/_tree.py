"""Attention for trees of drafts in 64 bits, from its definition; the bound on
the kernel's error is the one that _attn.py derives."""
import math

import numpy as np
import torch

from _attn import half_step


def sees(mask, rows, n):
    """[n, n] bool: draft i (a row of the mask) sees draft j."""
    words = mask[rows].cpu().numpy().view(np.uint32).astype(np.int64)
    out = np.zeros((n, n), bool)
    for j in range(min(n, 32 * words.shape[1])):
        out[:, j] = (words[:, j // 32] >> (j % 32)) & 1
    return out


def reference(q, k, v, table, start, lens, mask, scale, window=0, sinks=0):
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
        tree = sees(mask, rows, n)
        before = L - n
        pos = before - 1 + tree.sum(1)
        key = np.arange(max(L, 1))
        seen = np.broadcast_to((key < before)[None], (n, len(key))).copy()
        if window:
            seen &= (key[None] > pos[:, None] - window) | (key[None] < sinks)
        for j in range(n):
            if 0 <= before + j < L:
                seen[:, before + j] = tree[:, j]
        seen &= (key < L)[None]
        used = torch.from_numpy(seen.any(0))
        seen = torch.from_numpy(seen).to(dev)
        key = torch.from_numpy(key)
        page = table[b][key // P]
        ok = (page >= 0) & (page < pages)
        bad = (used & ~ok).to(dev)
        take = torch.where(ok & used, page, 0).to(dev)
        slot = (key % P).to(dev)
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


def words_of(rows, words):
    """Python integers of bits as int32 words [len(rows), words]."""
    a = np.array([[(x >> 32 * w) & 0xffffffff for w in range(words)] for x in rows], np.uint32)
    return torch.from_numpy(a.reshape(len(rows), words).view(np.int32)).cuda()


def random_tree(n, r, wide=4):
    """Bits of a draft and those above it, for n drafts."""
    up = []
    for i in range(n):
        parent = i - 1 - int(r.randint(0, wide))
        up.append((up[parent] if parent >= 0 else 0) | 1 << i)
    return up


class Trees:
    """Random inputs: lists of drafts and context lengths (drafts included), pages
    shuffled over a pool; whatever no row sees is poisoned.  masks: "tree", "any"
    (bits at random, some rows empty, bits behind the drafts set too) or "chain"."""

    def __init__(self, drafts, ctx, heads, kv, dim=128, page=64, dtype=torch.bfloat16, seed=0,
                 window=0, sinks=0, masks="tree", words=None, extra_rows=0, max_context=None,
                 poison=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = np.random.RandomState(seed)
        B = len(drafts)
        self.window, self.sinks, self.scale = window, sinks, dim ** -0.5
        self.max_context = max(ctx) if max_context is None else max_context
        cols = max(1, -(-self.max_context // page))
        words = -(-max(drafts + [1]) // 32) if words is None else words
        T = sum(drafts) + extra_rows
        rows = []
        for n in drafts:
            if masks == "tree":
                rows += random_tree(n, r)
            elif masks == "chain":
                rows += [(2 << i) - 1 for i in range(n)]
            else:
                rows += [int.from_bytes(r.bytes(4 * words), "little") if r.rand() < 0.8 else 0
                         for _ in range(n)]
        rows += [0] * extra_rows
        self.mask = words_of(rows, words) if words else torch.zeros(T, 0, dtype=torch.int32,
                                                                    device="cuda")
        self.start = torch.tensor([0] + list(np.cumsum(drafts)), dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        clamped = [min(c, self.max_context) for c in ctx]
        table = np.full((B, cols), -1, np.int64)
        need = [(b, j) for b in range(B) for j in range(-(-clamped[b] // page))]
        pool = len(need) + 2
        perm = r.permutation(pool)
        seen = np.zeros((pool, page), bool)
        at = 0
        visible = []
        for b in range(B):
            n, L = drafts[b], clamped[b]
            tree = sees(self.mask, slice(at, at + n), n) if n else np.zeros((0, 0), bool)
            at += n
            before = L - n
            key = np.arange(cols * page)
            low = max(0, before - window + int(tree.sum(1).min())) if window and n else 0
            vis = (key < before) & ((key >= low) | (key < sinks)) & (n > 0)
            for j in range(n):
                if before + j >= 0:
                    vis[before + j] = tree[:, j].any()
            visible.append(vis & (key < L))
        for i, (b, j) in enumerate(need):
            vis = visible[b][j * page:(j + 1) * page]
            if vis.any():
                table[b, j] = perm[i]
                seen[perm[i]] = vis
            elif drafts[b] and (j + 1) * page > clamped[b] - drafts[b] - window:
                table[b, j] = perm[i]  # may be loaded: drafts that no mask names
            else:
                table[b, j] = r.choice([-1, pool, 2 ** 31 - 1, -(2 ** 31)])  # never read
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
        self.q = rand(T, heads, dim) * 2
        self.k, self.v = rand(pool, page, kv, dim), rand(pool, page, kv, dim)
        if poison:
            dead = torch.from_numpy(~seen).cuda()
            junk = torch.tensor([math.nan, math.inf, -math.inf, 3e4], dtype=dtype, device="cuda")
            self.k[dead] = junk[torch.arange(int(dead.sum()), device="cuda") % 4][:, None, None]
            self.v[dead] = junk[torch.arange(int(dead.sum()), device="cuda") % 3][:, None, None]
        self.table = torch.from_numpy(table).to(torch.int32).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, **kw):
        import prep_token_gb300 as dp
        return dp.dsa_tree_attention(self.q, self.k, self.v, self.table, self.start, self.lens,
                                     self.max_context, self.mask, scale=self.scale,
                                     window=self.window, sinks=self.sinks, err_flags=self.err, **kw)

    def check(self, out, lse):
        lens = torch.clamp(self.lens, max=self.max_context)
        want, z, tol, tol_l = reference(self.q, self.k, self.v, self.table, self.start, lens,
                                        self.mask, self.scale, self.window, self.sinks)
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
