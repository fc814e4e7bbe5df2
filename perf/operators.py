"""The paged-cache operators as a serving loop uses them: attention of new
tokens over a paged K/V cache (whole context, or a sliding window with the
first tokens kept visible), and the upkeep of the cache's pages (copy, fork
and free, compact).

`run` computes a case in its plain form, or, where `own` is true, through the
framework's calls.  A sequence's lengths belong to the case; the values, the
order of the pages and the pool's holes come from the seed.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
INDEX_ROW = 132  # bytes of a slot of the index-K cache: 128 codes and a scale


# ------------------------------------------------------------------- cases

def _attend(name, dtype, batch, heads, kv_heads, dim, page, new, context, window=0, sinks=0,
            ragged=False):
    c = dict(op="attend", dtype=dtype, batch=batch, heads=heads, kv_heads=kv_heads, dim=dim,
             page=page, new=new, context=context, window=window, sinks=sinks, ragged=ragged)
    return dict(c, name=name) if name else c


def _pages(name, op, caches, pool, page_bytes, **more):
    c = dict(op=op, caches=caches, pool=pool, page_bytes=page_bytes, **more)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request, one token, a context under the indexer's top-k: latency
        _attend("decode 1 x 1000", "bf16", 1, 64, 8, 128, 64, 1, 1000),
        # a decode step of 64 requests whose contexts differ
        _attend("decode 64 x 8192 ragged", "bf16", 64, 64, 8, 128, 64, 1, 8192, ragged=True),
        # one request with a long context: few rows, split over the keys
        _attend("decode 2 x 65536 fp16", "fp16", 2, 32, 4, 128, 64, 1, 65536),
        # a chunk of a long prompt behind a cached prefix
        _attend("chunk 2048 over 16384", "bf16", 1, 64, 8, 128, 64, 2048, 16384),
        # a mixed batch: ragged chunks, an idle slot, small pages, no shared heads
        _attend("mixed 12 chunks fp16 d64", "fp16", 12, 16, 16, 64, 16, 700, 4000, ragged=True),
        # sliding-window layers: a whole prompt, and a decode step whose old pages are gone
        _attend("window 1024 prompt 8192", "bf16", 1, 32, 8, 128, 64, 8192, 8192, 1024, 16),
        _attend("window 4096 decode 32", "bf16", 32, 32, 4, 128, 64, 1, 131072, 4096, 4, True),
        # page copies: a handful of index-K pages of 21 layers; a prefix's worth of K/V pages
        _pages("copy 16 pages x 21", "copy", 21, 1024, 64 * INDEX_ROW, pages=16),
        _pages("copy 1024 pages x 4", "copy", 4, 2304, 64 * 8 * 128 * 2, pages=1024),
        # a search that branches: children share their parents' whole pages, then go
        _pages("fork 4 of 1, free", "fork", 21, 1024, 64 * INDEX_ROW, page=64, parents=1,
               children=4, context=1000, table=64),
        _pages("fork 64 of 8, free", "fork", 8, 2304, 64 * 8 * 128 * 2, page=64, parents=8,
               children=64, context=16300, table=512),
        # a pool three quarters empty is packed so that its upper part can be given back
        _pages("compact 2048 x 8", "compact", 8, 2048, 64 * 8 * 128 * 2, page=64, rows=48,
               live=600, table=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "chunk", "chunk", "window", "window", "copy", "fork",
                       "compact"])
    if kind in ("decode", "chunk", "window"):
        dtype = rng.choice(["bf16", "fp16"])
        dim = rng.choice([64, 128, 128])
        page = rng.choice([16, 32, 64, 64, 128])
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 5, 8, 8])
        window = sinks = 0
        ragged = rng.random() < 0.6
        if kind == "decode":
            context = _log_int(rng, 1, 60000)
            batch = _log_int(rng, 1, max(1, min(200, 2_000_000 // (context * kv))))
            new = rng.choice([1, 1, 1, 2, 5])
        elif kind == "chunk":
            context = _log_int(rng, 64, 12000)
            new = _log_int(rng, 2, min(context, 3000))
            batch = _log_int(rng, 1, max(1, min(32, 300_000_000 // (context * new * kv * group))))
        else:
            window = _log_int(rng, 1, 5000)
            sinks = rng.choice([0, 1, 4, 16, 100])
            context = _log_int(rng, 200, 100000)
            new = rng.choice([1, 1, _log_int(rng, 2, 2000)])
            batch = _log_int(rng, 1, max(1, min(
                48, 300_000_000 // ((window + new + 128) * max(new, 64) * kv * group))))
        return _attend(None, dtype, batch, kv * group, kv, dim, page, min(new, context), context,
                       window, sinks, ragged)
    page = rng.choice([16, 32, 64])
    bytes_ = page * rng.choice([INDEX_ROW, 512, 1024, 2048])
    caches = rng.randint(1, 24)
    most = max(64, min(4096, 600_000_000 // (caches * bytes_)))
    pool = rng.randint(most // 2, most)
    if kind == "copy":
        return _pages(None, "copy", caches, pool, bytes_, pages=_log_int(rng, 1, pool // 3))
    if kind == "fork":
        parents = rng.randint(1, 4)
        children = _log_int(rng, 1, max(1, pool // 8))
        blocks = max(1, pool // (2 * parents))
        context = _log_int(rng, 1, blocks * page)
        return _pages(None, "fork", caches, pool, bytes_, page=page, parents=parents,
                      children=min(children, 100), context=context, table=blocks + rng.randint(1, 9))
    live = _log_int(rng, 1, pool - 1)
    rows = rng.randint(1, 40)
    return _pages(None, "compact", caches, pool, bytes_, page=page, rows=rows, live=live,
                  table=-(-live // rows) + rng.randint(1, 9))


def _lengths(c):
    """New tokens and context (new ones included) of each sequence: the case's own."""
    B, new, ctx = c["batch"], c["new"], c["context"]
    if not c["ragged"]:
        return np.full(B, new, np.int64), np.full(B, ctx, np.int64)
    r = np.random.RandomState(B * 7919 + ctx)
    n = r.randint(1, new + 1, B)
    length = np.maximum(n, r.randint(max(1, ctx // 16), ctx + 1, B))
    n[0], length[0] = new, ctx
    if B >= 4 and new > 1:
        n[1] = length[1] = 0  # an idle slot of the batch
    return n.astype(np.int64), length.astype(np.int64)


def _visible_pairs(c):
    """(query, key) pairs that see each other, and keys that some query sees, for one head."""
    pairs = keys = 0
    w, s = c["window"], c["sinks"]
    for n, L in zip(*_lengths(c)):
        pos = np.arange(L - n, L)
        lo = np.maximum(0, pos - w + 1) if w else np.zeros_like(pos)
        pairs += int((pos + 1 - lo + np.minimum(lo, s)).sum())
        if n:
            keys += int(L - lo[0] + min(int(lo[0]), s))
    return pairs, keys


def work(c):
    if c["op"] == "attend":
        pairs, keys = _visible_pairs(c)
        T = int(_lengths(c)[0].sum())
        return {"bytes": 2 * (2 * T * c["heads"] * c["dim"] + 2 * keys * c["kv_heads"] * c["dim"])
                + 4 * T * c["heads"], "flops": 4 * c["dim"] * c["heads"] * pairs}
    if c["op"] == "copy":
        return {"bytes": 2 * c["pages"] * c["caches"] * c["page_bytes"] + 8 * c["pages"], "flops": 0}
    if c["op"] == "fork":  # a parent's last page is read once, whatever the number of its children
        blocks = -(-c["context"] // c["page"])
        part = 1 if c["context"] % c["page"] else 0
        moved = part * (min(c["parents"], c["children"]) + c["children"])
        return {"bytes": moved * c["caches"] * c["page_bytes"] + 4 * c["pool"]
                + 16 * blocks * c["children"], "flops": 0}
    live, pool = c["live"], c["pool"]
    moved = live - live * live // pool  # expected, for pages spread evenly over the pool
    return {"bytes": 2 * moved * c["caches"] * c["page_bytes"] + 8 * pool + 8 * live, "flops": 0}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def prepare(c, seed):
    g = _generator(seed)
    return _prepare_attend(c, g) if c["op"] == "attend" else _prepare_pages(c, g, seed)


def _prepare_attend(c, g):
    n, length = _lengths(c)
    B, P, dt = c["batch"], c["page"], DTYPES[c["dtype"]]
    first = np.zeros(B, np.int64)  # pages of the window's past are gone, those of the sinks stay
    kept = np.zeros(B, np.int64)
    if c["window"]:
        first = np.maximum(0, length - np.maximum(n, 1) - c["window"] + 1) // P
        kept = np.minimum(first, -(-c["sinks"] // P))
    blocks = -(-length // P)
    width = max(1, -(-c["context"] // P))
    col = np.arange(width)[None]
    held = (col < blocks[:, None]) & ((col >= first[:, None]) | (col < kept[:, None]))
    pool = int(held.sum()) + 3
    shape = (pool, P, c["kv_heads"], c["dim"])
    k = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    v = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    T = int(n.sum())
    q = torch.randn((T, c["heads"], c["dim"]), generator=g, device="cuda", dtype=dt) * 2
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(pool, generator=g, device="cuda")[: pool - 3].to(torch.int32)
    table[torch.from_numpy(held).cuda()] = order
    start = np.concatenate([[0], np.cumsum(n)])
    return dict(case=c, q=q, k=k, v=v, table=table, max_query=int(n.max()),
                start=torch.from_numpy(start.astype(np.int32)).cuda(),
                lens=torch.from_numpy(length.astype(np.int32)).cuda(),
                scale=c["dim"] ** -0.5)


def _prepare_pages(c, g, seed):
    N, pb = c["pool"], c["page_bytes"]
    caches = torch.randint(-(2 ** 31), 2 ** 31 - 1, (c["caches"], N, pb // 4), generator=g,
                           device="cuda", dtype=torch.int32)
    s = dict(case=c, all=caches, caches=list(caches.unbind(0)))
    perm = torch.randperm(N, generator=g, device="cuda")
    if c["op"] == "copy":
        s["src"], s["dst"] = (perm[i * c["pages"]:(i + 1) * c["pages"]].to(torch.int32)
                              for i in (0, 1))
        return s
    if c["op"] == "fork":
        n, m, P = c["parents"], c["children"], c["page"]
        blocks = -(-c["context"] // P)
        table = torch.full((n + m, c["table"]), -1, dtype=torch.int32, device="cuda")
        table[:n, :blocks] = perm[: n * blocks].view(n, blocks).to(torch.int32)
        lens = torch.zeros(n + m, dtype=torch.int32, device="cuda")
        lens[:n] = c["context"]
        refs = torch.zeros(N, dtype=torch.int32, device="cuda")
        refs[perm[: n * blocks]] = 1
        s.update(table=table, lens=lens, refs=refs,
                 parents=torch.randint(0, n, (m,), generator=g, device="cuda", dtype=torch.int32),
                 children=(n + torch.randperm(m, generator=g, device="cuda")).to(torch.int32))
        return s
    R, P, live = c["rows"], c["page"], c["live"]
    share = np.bincount(np.arange(live) % R, minlength=R)  # pages of each row
    tail = np.random.RandomState(seed % (1 << 31)).randint(1, P + 1, R)
    lens = np.where(share > 0, (share - 1) * P + tail, 0).astype(np.int32)
    held = np.arange(c["table"])[None] < share[:, None]
    table = torch.full((R, c["table"]), -1, dtype=torch.int32, device="cuda")
    table[torch.from_numpy(held).cuda()] = perm[:live].to(torch.int32)
    refs = torch.zeros(N, dtype=torch.int32, device="cuda")
    refs[perm[:live]] = 1
    s.update(table0=table, refs0=refs, table=table.clone(), refs=refs.clone(),
             lens=torch.from_numpy(lens).cuda())
    return s


# --------------------------------------------------------------- one pass

def run(s):
    return {"attend": _run_attend, "copy": _run_copy, "fork": _run_fork,
            "compact": _run_compact}[s["case"]["op"]](s)


def _run_attend(s):
    c = s["case"]
    if own:
        import prep_token_gb300 as dp
        out, lse = dp.dsa_paged_attention(
            s["q"], s["k"], s["v"], s["table"], s["start"], s["lens"], c["context"],
            scale=s["scale"], window=c["window"], sinks=c["sinks"])
        return {"out": out, "lse": lse}
    # The queries padded to [B, Q], the keys that any of them can see gathered
    # to [B, W]: the last window + Q - 1 of the context and the sinks.
    q, start, lens = s["q"], s["start"].long(), s["lens"].long()
    B, Q, P, D, kv = c["batch"], s["max_query"], c["page"], c["dim"], c["kv_heads"]
    G, T = c["heads"] // kv, q.shape[0]
    dev = q.device
    w, sinks = c["window"] or c["context"], c["sinks"] if c["window"] else 0
    n = start[1:] - start[:-1]
    i = torch.arange(Q, device=dev)
    pos = (lens - n)[:, None] + i                                            # [B, Q]
    reach = min(c["context"], w + Q - 1)
    base = (lens - reach).clamp(min=0)
    key = torch.cat([torch.arange(min(sinks, c["context"]), device=dev).expand(B, -1),
                     base[:, None] + torch.arange(reach, device=dev)], 1)    # [B, W]
    once = torch.arange(key.shape[1], device=dev) >= sinks                   # not a sink twice
    there = (key < lens[:, None]) & (~once | (key >= sinks) | (sinks == 0))
    page = s["table"].long().gather(1, (key // P).clamp(max=s["table"].shape[1] - 1))
    there = there & (page >= 0)
    slot = page.clamp(min=0) * P + key % P
    k = s["k"].view(-1, kv, D)[slot].float().permute(0, 2, 3, 1)             # [B, kv, D, W]
    v = s["v"].view(-1, kv, D)[slot].float().masked_fill(~there[..., None, None], 0)
    qp = q[(start[:-1, None] + i).clamp(max=T - 1)].float() * s["scale"]     # [B, Q, H, D]
    qp = qp.view(B, Q, kv, G, D).permute(0, 2, 3, 1, 4).reshape(B, kv, G * Q, D)
    score = (qp @ k).view(B, kv, G, Q, -1)
    seen = there[:, None] & (key[:, None] <= pos[..., None]) & (
        (key[:, None] > pos[..., None] - w) | (key[:, None] < sinks))        # [B, Q, W]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = score.view(B, kv, G * Q, -1) @ v.transpose(1, 2)
    out = out.view(B, kv, G, Q, D) / total.clamp(min=1e-38)
    lse = torch.where(total > 0, top + total.log(), -math.inf)[..., 0]
    row = torch.arange(T, device=dev)
    b = torch.searchsorted(start[1:].contiguous(), row, right=True)
    at = row - start[b]
    return {"out": out.permute(0, 3, 1, 2, 4).reshape(B, Q, c["heads"], D)[b, at].to(q.dtype),
            "lse": lse.permute(0, 3, 1, 2).reshape(B, Q, c["heads"])[b, at]}


def _run_copy(s):
    if own:
        import prep_token_gb300 as dp
        dp.dsa_cache_copy_pages(s["caches"], s["case"]["pool"], s["src"], s["dst"])
    else:
        s["all"][:, s["dst"].long()] = s["all"][:, s["src"].long()]
    return {"caches": s["all"]}


def _run_fork(s):
    """Children forked, the rows that the next attention call takes, the children freed."""
    c, table, lens, refs = s["case"], s["table"], s["lens"], s["refs"]
    P, children = c["page"], s["children"].long()
    if own:
        import prep_token_gb300 as dp
        dp.dsa_cache_fork(s["caches"], refs, table, lens, P, s["parents"], s["children"])
        rows, length = table[children], lens[children]
        dp.dsa_cache_free(refs, table, lens, P, s["children"])
        return {"caches": s["all"], "rows": rows, "length": length, "refs": refs, "table": table,
                "lens": lens}
    parents = s["parents"].long()
    L = lens[parents].long()
    whole, part = L // P, L % P > 0
    lowest = torch.argsort((refs != 0).int(), stable=True)  # the free pages, lowest first
    fresh = lowest[(part.long().cumsum(0) - 1).clamp(min=0)]
    col = torch.arange(table.shape[1], device=refs.device)[None]
    rows = torch.where(col < whole[:, None], table[parents], -1)
    rows = torch.where((col == whole[:, None]) & part[:, None], fresh[:, None].int(), rows)
    old = table[parents].gather(1, whole.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
    into = torch.where(part, fresh, old.clamp(min=0))
    s["all"][:, into] = s["all"][:, torch.where(part, old, into)]
    held = (rows >= 0).int().view(-1)
    refs.index_add_(0, rows.view(-1).long().clamp(min=0), held)
    table[children] = rows
    lens[children] = L.int()
    rows, length = table[children], lens[children]
    # free
    drop = table[children]
    refs.index_add_(0, drop.view(-1).long().clamp(min=0), -(drop >= 0).int().view(-1))
    table[children] = -1
    lens[children] = 0
    return {"caches": s["all"], "rows": rows, "length": length, "refs": refs, "table": table,
            "lens": lens}


def _run_compact(s):
    """The pool's tables are put back as they were first, so that each pass packs the same pool."""
    c = s["case"]
    refs, table = s["refs"].copy_(s["refs0"]), s["table"].copy_(s["table0"])
    if own:
        import prep_token_gb300 as dp
        live = dp.dsa_cache_compact(s["caches"], refs, table, s["lens"], c["page"])
        return {"caches": s["all"], "refs": refs, "table": table, "live": live}
    used = refs > 0
    live = used.sum()
    at = torch.arange(c["pool"], device=refs.device)
    src = (used & (at >= live)).nonzero()[:, 0]
    dst = (~used & (at < live)).nonzero()[:, 0]
    s["all"][:, dst] = s["all"][:, src]
    to = at.clone()
    to[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, to[table.long().clamp(min=0)].int(), table))
    return {"caches": s["all"], "refs": refs, "table": table, "live": live.int().view(1)}


# ---------------------------------------------------------- the definition

def exact(c, seed):
    s = prepare(c, seed)
    return _exact_attend(c, s) if c["op"] == "attend" else _exact_pages(c, s)


def _exact_attend(c, s):
    """Sequence by sequence and kv head by kv head, in 64 bits: a softmax over the visible keys."""
    T, H, D = s["q"].shape
    P, kv, w, sinks = c["page"], c["kv_heads"], c["window"], c["sinks"]
    G = H // kv
    out = torch.zeros((T, H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    start = 0
    for b, (n, L) in enumerate(zip(*(x.tolist() for x in _lengths(c)))):
        if not n:
            continue
        low = max(0, L - n - w + 1) if w else 0
        keys = [j for j in range(0, min(sinks, low))] + list(range(low, L))
        keys = torch.tensor(keys, device="cuda")
        pages = s["table"][b].long()[torch.div(keys, P, rounding_mode="floor")]
        pos = torch.arange(L - n, L, device="cuda")[:, None]
        hidden = keys[None] > pos
        if w:
            hidden |= (keys[None] <= pos - w) & (keys[None] >= sinks)
        for h in range(kv):
            K = s["k"][pages, keys % P, h].double()
            V = s["v"][pages, keys % P, h].double()
            for i in range(0, n, 1024):
                rows = slice(start + i, start + min(n, i + 1024))
                Q = s["q"][rows, h * G:(h + 1) * G].double()
                x = torch.einsum("tgd,kd->tgk", Q, K) * s["scale"]
                x.masked_fill_(hidden[i:i + 1024][:, None], -math.inf)
                z = torch.logsumexp(x, -1)
                lse[rows, h * G:(h + 1) * G] = z
                out[rows, h * G:(h + 1) * G] = torch.einsum("tgk,kd->tgd", (x - z[..., None]).exp(), V)
        start += n
    return {"out": out, "lse": lse}


def _exact_pages(c, s):
    """The bookkeeping, page by page on the host (the caches' bytes have no other form)."""
    if c["op"] == "copy":
        return None
    if c["op"] == "fork":
        P = c["page"]
        refs, table, lens = s["refs"].tolist(), s["table"].tolist(), s["lens"].tolist()
        rows, length = [], []
        free = iter([p for p, r in enumerate(refs) if r == 0])
        for a in s["parents"].tolist():
            L = lens[a]
            row = table[a][: L // P] + ([next(free)] if L % P else [])
            rows.append(row + [-1] * (c["table"] - len(row)))
            length.append(L)
        as_int = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
        return {"caches": None, "rows": as_int(rows), "length": as_int(length),
                "refs": as_int(refs), "table": as_int(table), "lens": as_int(lens)}
    refs, table = s["refs0"].tolist(), s["table0"].tolist()
    live = sum(r > 0 for r in refs)
    moved = [p for p in range(live, c["pool"]) if refs[p]]
    holes = [p for p in range(live) if not refs[p]]
    to = dict(zip(moved, holes))
    for a, b in to.items():
        refs[b], refs[a] = refs[a], 0
    table = [[to.get(p, p) for p in row] for row in table]
    return {"caches": None, "refs": torch.tensor(refs, dtype=torch.int32),
            "table": torch.tensor(table, dtype=torch.int32),
            "live": torch.tensor([live], dtype=torch.int32)}
