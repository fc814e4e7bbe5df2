"""The operators of a step that verifies drafted tokens, as a serving loop uses
them next to the paged attention and the pages' upkeep: the norm in front of a
layer's projections (with the residual's addition, in 16 bits or in e4m3 with
scales), the rotation of q and k with K and V appended to the paged cache,
attention for a tree of drafted tokens, and the accepted drafts' entries moved
to where they belong.  Norm and append serve prompts and plain decoding too.

`run` computes a case in its plain form, or, where `own` is true, through the
framework's calls.  A sequence's lengths belong to the case; the values, the
trees and the order of the pages come from the seed.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
MAX_POSITION = 40960


# ------------------------------------------------------------------- cases

def _case(name, op, **c):
    c = dict(c, op=op)
    return dict(c, name=name) if name else c


def _norm(name, dtype, tokens, width, residual=True, out="fp8", group=128):
    return _case(name, "norm", dtype=dtype, tokens=tokens, width=width, residual=residual, out=out,
                 group=group)


def _append(name, dtype, tokens, heads, kv_heads, dim, page, rope, style="neox", norm=False):
    return _case(name, "append", dtype=dtype, tokens=tokens, heads=heads, kv_heads=kv_heads,
                 dim=dim, page=page, rope=rope, style=style, norm=norm)


def _tree(name, dtype, batch, heads, kv_heads, dim, page, drafts, context, window=0, sinks=0,
          ragged=False):
    return _case(name, "tree", dtype=dtype, batch=batch, heads=heads, kv_heads=kv_heads, dim=dim,
                 page=page, drafts=drafts, context=context, window=window, sinks=sinks,
                 ragged=ragged)


def _keep(name, layers, batch, kv_heads, dim, page, drafts, context):
    return _case(name, "keep", layers=layers, batch=batch, kv_heads=kv_heads, dim=dim, page=page,
                 drafts=drafts, context=context)


def listed():
    return [
        # the norm of one request's token in a decode step: latency
        _norm("norm 1 x 7168 to fp8", "bf16", 1, 7168),
        # the last norm of a ragged batch, for a head that takes 16 bits
        _norm("norm 777 x 5120 fp16", "fp16", 777, 5120, out="16"),
        # a large prompt batch in front of fp8 projections
        _norm("norm 16384 x 7168 to fp8", "bf16", 16384, 7168),
        # one step's new tokens of 16 requests: latency
        _append("append 16 tokens", "bf16", 16, 64, 8, 128, 64, 64, "gptj"),
        # a prompt's tokens, in a model with q and k norms
        _append("append 8192 with norms", "bf16", 8192, 32, 8, 128, 64, 128, "neox", True),
        # a mixed batch, small pages, no shared heads
        _append("append 1500 fp16 d64", "fp16", 1500, 24, 24, 64, 16, 32),
        # one request's short chainlike tree: latency
        _tree("tree 1 x 8 over 1000", "bf16", 1, 64, 8, 128, 64, 8, 1000),
        # a full batch of small trees whose contexts differ
        _tree("tree 64 x 16 over 8192 ragged", "bf16", 64, 64, 8, 128, 64, 16, 8192, ragged=True),
        # few requests, wide trees, long contexts: few rows, split over the keys
        _tree("tree 4 x 60 over 32768 fp16", "fp16", 4, 32, 4, 128, 64, 60, 32768),
        # a sliding-window layer, small pages, no shared heads
        _tree("tree window 1024 24 x 32 d64", "bf16", 24, 16, 16, 64, 16, 32, 30000, 1024, 4, True),
        # the accepted path of one request in 21 layers: latency
        _keep("keep 1 of 21 layers", 21, 1, 8, 128, 64, 8, 1000),
        # a full batch's accepted paths in every layer's K and V
        _keep("keep 48 of 40 layers", 40, 48, 8, 128, 64, 32, 90),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "append", "append", "tree", "tree", "tree", "keep"])
    dtype = rng.choice(["bf16", "fp16"])
    dim = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 64, 128])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8, 8])
    if kind == "norm":
        width = 8 * _log_int(rng, 8, 2048)
        tokens = _log_int(rng, 1, min(20000, 110_000_000 // width))
        return _norm(None, dtype, tokens, width, rng.random() < 0.7, rng.choice(["fp8", "fp8", "16"]),
                     rng.choice([32, 128, 128]))
    if kind == "append":
        tokens = _log_int(rng, 1, min(12000, 48_000_000 // ((kv * group + 2 * kv) * dim)))
        return _append(None, dtype, tokens, kv * group, kv, dim, page,
                       16 * rng.randint(0, dim // 16), rng.choice(["neox", "gptj"]),
                       rng.random() < 0.5)
    if kind == "tree":
        window = rng.choice([0, 0, _log_int(rng, 30, 4000)])
        context = _log_int(rng, 100, 60000)
        drafts = min(context, rng.choice([1, 5, 8, 16, 33, 64, _log_int(rng, 2, 150)]))
        reach = min(context, window + drafts) if window else context
        batch = _log_int(rng, 1, max(1, min(100, 2_000_000 // (reach * kv),
                                            180_000_000 // (reach * drafts * kv * group))))
        return _tree(None, dtype, batch, kv * group, kv, dim, page, drafts, context, window,
                     rng.choice([0, 4, 50]) if window else 0, rng.random() < 0.6)
    batch = _log_int(rng, 1, 64)
    context = _log_int(rng, 1, 200)
    drafts = rng.randint(1, 40)
    pages = batch * (-(-(context + drafts) // page))
    most = max(1, min(48, 1_500_000_000 // (pages * page * kv * dim * 4)))
    return _keep(None, rng.randint(1, most), batch, kv, dim, page, drafts, context)


def _lengths(c):
    """Drafted tokens and context (drafts included) of each sequence: the case's own."""
    B, new, ctx = c["batch"], c["drafts"], c["context"]
    if not c["ragged"]:
        return np.full(B, new, np.int64), np.full(B, ctx, np.int64)
    r = np.random.RandomState(B * 7919 + ctx)
    n = r.randint(1, new + 1, B)
    length = np.maximum(n, r.randint(max(1, ctx // 16), ctx + 1, B))
    n[0], length[0] = new, ctx
    if B >= 4:
        n[1] = length[1] = 0  # an idle slot of the batch
    return n.astype(np.int64), length.astype(np.int64)


def _accepted(c):
    """Of each sequence: tokens before the drafts, drafts, and the accepted ones, ascending."""
    r = np.random.RandomState(c["batch"] * 101 + c["drafts"])
    for _ in range(c["batch"]):
        d = int(r.randint((c["drafts"] + 1) // 2, c["drafts"] + 1))
        k = int(r.randint(0, min(d, 8) + 1))
        yield int(r.randint((c["context"] + 1) // 2, c["context"] + 1)), d, np.sort(
            r.choice(d, k, replace=False))


def work(c):
    if c["op"] == "norm":
        each = 2 + (4 if c["residual"] else 0) + (1 + 1 / c["group"] if c["out"] == "fp8" else 2)
        return {"bytes": each * c["tokens"] * c["width"] + 4 * c["width"],
                "flops": 4 * c["tokens"] * c["width"]}
    if c["op"] == "append":
        rows = c["tokens"] * (c["heads"] + 2 * c["kv_heads"])
        return {"bytes": 4 * rows * c["dim"] + c["tokens"] * (16 + 4 * c["rope"]),
                "flops": 3 * rows * c["dim"]}
    if c["op"] == "tree":
        n, length = _lengths(c)
        before = length - n
        seen = before if not c["window"] else np.minimum(before, c["window"] + c["sinks"])
        pairs = int((n * seen + n * (n + 1) // 2).sum())  # at most: a chain
        keys, T = int((seen + n).sum()), int(n.sum())
        return {"bytes": 2 * (2 * T * c["heads"] * c["dim"] + 2 * keys * c["kv_heads"] * c["dim"])
                + 4 * T * c["heads"], "flops": 4 * c["dim"] * c["heads"] * pairs}
    moved = sum(int((k != np.arange(len(k))).sum()) for _, _, k in _accepted(c))
    return {"bytes": 2 * moved * c["layers"] * 2 * c["kv_heads"] * c["dim"] * 2
            + 64 * c["batch"], "flops": 0}


# ------------------------------------------------------------------ inputs

def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"norm": _prepare_norm, "append": _prepare_append, "tree": _prepare_tree,
            "keep": _prepare_keep}[c["op"]](c, g, np.random.RandomState(seed % (1 << 31)))


def _prepare_norm(c, g, r):
    shape, dt = (c["tokens"], c["width"]), DTYPES[c["dtype"]]
    x = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    # a residual stream: larger than what is added, with a few channels that stick out
    res = torch.randn(shape, generator=g, device="cuda", dtype=dt) * 3
    res[:, :: max(1, c["width"] // 7)] *= 20
    gamma = torch.rand(c["width"], generator=g, device="cuda") + 0.5
    return dict(case=c, x=x, res=res if c["residual"] else None, gamma=gamma)


def _prepare_append(c, g, r):
    T, H, kv, D, P, dt = (c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["page"],
                          DTYPES[c["dtype"]])
    qkv = torch.randn((T, (H + 2 * kv) * D), generator=g, device="cuda", dtype=dt)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([H * D, kv * D, kv * D], 1))
    pages = -(-T // P) + 8
    page = torch.randperm(pages, generator=g, device="cuda")
    at = torch.arange(T, device="cuda") + int(r.randint(0, P))
    slots = page[at // P] * P + at % P
    positions = at + int(r.randint(0, MAX_POSITION - T - P))
    freq = 10000.0 ** (-torch.arange(c["rope"] // 2, device="cuda", dtype=torch.float64) * 2
                       / max(1, c["rope"]))
    angle = torch.arange(MAX_POSITION, device="cuda", dtype=torch.float64)[:, None] * freq
    cache = torch.zeros((2, pages, P, kv, D), device="cuda", dtype=dt)
    gamma = torch.rand((2, D), generator=g, device="cuda") + 0.5
    return dict(case=c, q=q, k=k, v=v, slots=slots, positions=positions,
                cos=angle.cos().float(), sin=angle.sin().float(), k_cache=cache[0],
                v_cache=cache[1], q_gamma=gamma[0], k_gamma=gamma[1])


def _trees(n, words, r):
    """Random trees' masks: bit j of a row's words is set where draft j is the row's own token
    or above it.  Every draft hangs on the context or on an earlier draft, the later ones rather."""
    rows = []
    for m in n:
        up = []
        for i in range(m):
            parent = i - 1 - int(r.randint(0, 4))
            up.append((up[parent] if parent >= 0 else 0) | 1 << i)
        rows += up
    return np.array([[(x >> 32 * w) & 0xffffffff for w in range(words)] for x in rows],
                    np.uint32).reshape(-1, words).view(np.int32)


def _prepare_tree(c, g, r):
    n, length = _lengths(c)
    B, P, dt = c["batch"], c["page"], DTYPES[c["dtype"]]
    blocks = -(-length // P)
    width = max(1, -(-c["context"] // P))
    first, kept = np.zeros(B, np.int64), np.zeros(B, np.int64)
    if c["window"]:  # pages of the window's past are gone, those of the sinks stay
        first = np.maximum(0, length - n - c["window"]) // P
        kept = np.minimum(first, -(-c["sinks"] // P))
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
                mask=torch.from_numpy(_trees(n, -(-c["drafts"] // 32), r)).cuda(),
                scale=c["dim"] ** -0.5)


def _prepare_keep(c, g, r):
    B, P = c["batch"], c["page"]
    before, drafted, kept = zip(*_accepted(c))
    length = np.array(before) + np.array(drafted)
    blocks = -(-length // P)
    cols = int(blocks.max())
    pool = int(blocks.sum()) + 5
    held = np.arange(cols)[None] < blocks[:, None]
    table = np.full((B, cols), -1, np.int32)
    table[held] = r.permutation(pool)[: int(blocks.sum())]
    refs = np.zeros(pool, np.int32)
    refs[table[held]] = 1
    width = max(1, max(len(k) for k in kept))
    chosen = np.zeros((B, width), np.int32)
    for b, k in enumerate(kept):
        chosen[b, :len(k)] = k
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    # the tables side by side: put back by one copy before each pass
    tables = up(np.concatenate([refs, length, table.ravel()]))
    now = tables.clone()
    caches = torch.randint(-(2 ** 15), 2 ** 15, (2 * c["layers"], pool, P, c["kv_heads"], c["dim"]),
                           generator=g, device="cuda", dtype=torch.int16)
    s = dict(case=c, all=caches, tables0=tables, tables=now, refs=now[:pool],
             lens=now[pool:pool + B], table=now[pool + B:].view(B, cols),
             rows=torch.arange(B, dtype=torch.int32, device="cuda"), drafted=up(drafted),
             kept=up(chosen), n_kept=up([len(k) for k in kept]))
    s["caches"] = list(caches.unbind(0))
    if own:  # the description of the layers' caches, which a program makes once
        import prep_token_gb300 as dp
        s["caches"] = dp.TokenViews(s["caches"])
    return s


# --------------------------------------------------------------- one pass

def run(s):
    return {"norm": _run_norm, "append": _run_append, "tree": _run_tree,
            "keep": _run_keep}[s["case"]["op"]](s)


def _run_norm(s):
    """The e4m3 codes and their scales come back as numbers (tensors of 8-bit floating types)."""
    c, x, res = s["case"], s["x"], s["res"]
    if own:
        import prep_token_gb300 as dp
        if c["out"] == "16":
            got = dp.dsa_rms_norm(x, s["gamma"], EPS, residual=res)
            return {"out": got[0], "residual": got[1]} if res is not None else {"out": got}
        got = dp.dsa_rms_norm_fp8(x, s["gamma"], EPS, residual=res, group=c["group"],
                                  scale_dtype=torch.float8_e8m0fnu)
        return dict(zip(("codes", "scales", "residual"), got))
    z = x.float() if res is None else x.float() + res.float()
    y = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS) * s["gamma"]
    out = {} if res is None else {"residual": z.to(x.dtype)}
    if c["out"] == "16":
        return dict(out, out=y.to(x.dtype))
    T, N = y.shape
    groups = -(-N // c["group"])
    whole = y.new_zeros(T, groups * c["group"])
    whole[:, :N] = y
    amax = whole.view(T, groups, -1).abs().amax(-1).clamp(min=1e-4)
    m, e = torch.frexp(amax)                       # 448 = 0.875 * 2^9
    e = e - 9 + (m > 0.875).int()
    codes = torch.ldexp(whole.view(T, groups, -1), -e[..., None]).view(T, -1)[:, :N]
    return dict(out, codes=codes.to(torch.float8_e4m3fn),
                scales=(e + 127).to(torch.uint8).view(torch.float8_e8m0fnu))


def _run_append(s):
    c, D, r = s["case"], s["case"]["dim"], s["case"]["rope"]
    k_cache, v_cache = s["k_cache"], s["v_cache"]
    if own:
        import prep_token_gb300 as dp
        norms = dict(q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=EPS) if c["norm"] else {}
        q = dp.dsa_kv_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cos"], s["sin"],
                             k_cache, v_cache, rope_dim=r,
                             rope_style=dp.NEOX if c["style"] == "neox" else dp.GPTJ, **norms)
        return {"q": q, "k_cache": k_cache, "v_cache": v_cache}
    cos, sin = (t[s["positions"]][:, None] for t in (s["cos"], s["sin"]))

    def rotated(x, gamma):
        x = x.float()
        if c["norm"]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma
        y = x.clone()
        a, b = ((slice(0, r // 2), slice(r // 2, r)) if c["style"] == "neox"
                else (slice(0, r, 2), slice(1, r, 2)))
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., b] * cos + x[..., a] * sin
        return y.to(s["q"].dtype)

    k_cache.view(-1, c["kv_heads"], D)[s["slots"]] = rotated(s["k"], s["k_gamma"])
    v_cache.view(-1, c["kv_heads"], D)[s["slots"]] = s["v"]
    return {"q": rotated(s["q"], s["q_gamma"]), "k_cache": k_cache, "v_cache": v_cache}


def _run_tree(s):
    c = s["case"]
    if own:
        import prep_token_gb300 as dp
        out, lse = dp.dsa_tree_attention(
            s["q"], s["k"], s["v"], s["table"], s["start"], s["lens"], c["context"], s["mask"],
            scale=s["scale"], window=c["window"], sinks=c["sinks"])
        return {"out": out, "lse": lse}
    # The queries padded to [B, Q], the keys that any of them can see gathered to [B, W]: the
    # drafts, the window's reach before them, and the sinks.
    q, start, lens = s["q"], s["start"].long(), s["lens"].long()
    B, Q, P, D, kv = c["batch"], s["max_query"], c["page"], c["dim"], c["kv_heads"]
    G, T = c["heads"] // kv, q.shape[0]
    dev = q.device
    w, sinks = c["window"] or c["context"], c["sinks"] if c["window"] else 0
    n = start[1:] - start[:-1]
    before = lens - n
    i = torch.arange(Q, device=dev)
    row = (start[:-1, None] + i).clamp(max=T - 1)                            # [B, Q]
    bits = torch.arange(32, device=dev)
    mask = (s["mask"].long()[..., None] >> bits & 1).view(T, -1)[row] > 0    # [B, Q, 32 words]
    depth = (mask & (torch.arange(mask.shape[2], device=dev) < n[:, None, None])).sum(-1)
    pos = before[:, None] + depth - 1                                        # [B, Q]
    reach = min(c["context"], w + Q)
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
    qp = q[row].float() * s["scale"]                                         # [B, Q, H, D]
    qp = qp.view(B, Q, kv, G, D).permute(0, 2, 3, 1, 4).reshape(B, kv, G * Q, D)
    score = (qp @ k).view(B, kv, G, Q, -1)
    near = (key[:, None] > pos[..., None] - w) | (key[:, None] < sinks)
    draft = (key - before[:, None]).clamp(min=0, max=mask.shape[2] - 1)
    seen = torch.where((key < before[:, None])[:, None], near,
                       mask.gather(2, draft[:, None].expand(-1, Q, -1)))     # [B, Q, W]
    seen = seen & there[:, None]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = score.view(B, kv, G * Q, -1) @ v.transpose(1, 2)
    out = out.view(B, kv, G, Q, D) / total.clamp(min=1e-38)
    lse = torch.where(total > 0, top + total.log(), -math.inf)[..., 0]
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    at = t - start[b]
    return {"out": out.permute(0, 3, 1, 2, 4).reshape(B, Q, c["heads"], D)[b, at].to(q.dtype),
            "lse": lse.permute(0, 3, 1, 2).reshape(B, Q, c["heads"])[b, at]}


def _run_keep(s):
    """The pool's tables are put back as they were first, so that each pass keeps the same drafts."""
    c, P = s["case"], s["case"]["page"]
    s["tables"].copy_(s["tables0"])
    refs, lens, table = s["refs"], s["lens"], s["table"]
    if own:
        import prep_token_gb300 as dp
        dp.dsa_cache_keep(s["caches"], refs, table, lens, P, s["rows"], s["drafted"], s["kept"],
                          s["n_kept"])
        return {"caches": s["all"], "refs": refs, "lens": lens, "table": table}
    rows = s["rows"].long()
    before = (lens[rows] - s["drafted"]).long()[:, None]
    j = torch.arange(s["kept"].shape[1], device=refs.device)[None]
    some = j < s["n_kept"][:, None]
    tokens = table[rows].long()

    def slot(at):
        at = torch.where(some, at, 0)
        return (tokens.gather(1, at // P) * P + at % P)[some]

    src, dst = slot(before + s["kept"]), slot(before + j)
    flat = s["all"].flatten(1, 2)
    flat[:, dst] = flat[:, src]
    length = before[:, 0] + s["n_kept"]
    old = -(-lens[rows] // P)
    col = torch.arange(table.shape[1], device=refs.device)[None]
    gone = (col >= (-(-length // P))[:, None]) & (col < old[:, None]) & (tokens >= 0)
    refs.index_add_(0, tokens[gone], refs.new_full((), -1).expand(int(gone.sum())))
    table[rows] = torch.where(gone, -1, tokens).int()
    lens[rows] = length.int()
    return {"caches": s["all"], "refs": refs, "lens": lens, "table": table}


# ---------------------------------------------------------- the definition

def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "append": _exact_append, "tree": _exact_tree,
            "keep": _exact_keep}[c["op"]](c, s)


def _exact_norm(c, s):
    """Row blocks in 64 bits; an e4m3 code is the nearest of the 2^(e - 3) apart, ties to even."""
    out = {k: [] for k in ("out", "codes", "scales", "residual")}
    for i in range(0, c["tokens"], 2048):
        z = s["x"][i:i + 2048].double()
        if s["res"] is not None:
            z = z + s["res"][i:i + 2048].double()
            out["residual"].append(z)
        y = z / (z.pow(2).sum(-1, keepdim=True) / c["width"] + EPS).sqrt() * s["gamma"].double()
        if c["out"] == "16":
            out["out"].append(y)
            continue
        codes, scales = [], []
        for part in y.split(c["group"], 1):
            amax = part.abs().max(1, keepdim=True).values.clamp(min=1e-4)
            scale = torch.exp2(torch.ceil(torch.log2(amax / 448)))
            x = part / scale
            step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
            codes.append(torch.round(x / step) * step)
            scales.append(scale)
        out["codes"].append(torch.cat(codes, 1))
        out["scales"].append(torch.cat(scales, 1))
    return {k: torch.cat(v) for k, v in out.items() if v}


def _exact_append(c, s):
    """Pairs as complex numbers, turned by the angles' own."""
    D, r, T = c["dim"], c["rope"], c["tokens"]
    turn = torch.complex(s["cos"][s["positions"]].double(), s["sin"][s["positions"]].double())

    def rows(x, gamma):
        y = x.double()
        if c["norm"]:
            y = y / (y.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * gamma.double()
        pairs = y[..., :r].reshape(T, -1, 2, r // 2) if c["style"] == "neox" else \
            y[..., :r].reshape(T, -1, r // 2, 2).transpose(2, 3)
        z = torch.complex(pairs[:, :, 0].contiguous(), pairs[:, :, 1].contiguous()) * turn[:, None]
        z = torch.stack([z.real, z.imag], 2 if c["style"] == "neox" else 3)
        return torch.cat([z.reshape(T, -1, r), y[..., r:]], -1)

    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    page = torch.div(s["slots"], c["page"], rounding_mode="floor")
    k_cache[page, s["slots"] % c["page"]] = rows(s["k"], s["k_gamma"])
    v_cache[page, s["slots"] % c["page"]] = s["v"].double()
    return {"q": rows(s["q"], s["q_gamma"]), "k_cache": k_cache, "v_cache": v_cache}


def _exact_tree(c, s):
    """Sequence by sequence and kv head by kv head, in 64 bits: a softmax over the visible keys."""
    T, H, D = s["q"].shape
    P, kv, w, sinks = c["page"], c["kv_heads"], c["window"], c["sinks"]
    G = H // kv
    out = torch.zeros((T, H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    masks = s["mask"].cpu().numpy().view(np.uint32)
    start = 0
    for b, (n, L) in enumerate(zip(*(x.tolist() for x in _lengths(c)))):
        if not n:
            continue
        rows = slice(start, start + n)
        before = L - n
        words = masks[rows].astype(np.int64)
        sees = (words[:, np.arange(n) // 32] >> (np.arange(n) % 32)) & 1    # [n, drafts]
        pos = before + sees.sum(1) - 1
        low = max(0, before - w) if w else 0
        keys = np.concatenate([np.arange(min(sinks, low)), np.arange(low, L)])
        hidden = np.zeros((n, len(keys)), bool)
        if w:
            hidden |= (keys[None] <= pos[:, None] - w) & (keys[None] >= sinks)
        hidden[:, len(keys) - n:] = sees == 0
        hidden, keys = torch.from_numpy(hidden).cuda(), torch.from_numpy(keys).cuda()
        pages = s["table"][b].long()[torch.div(keys, P, rounding_mode="floor")]
        for h in range(kv):
            K = s["k"][pages, keys % P, h].double()
            V = s["v"][pages, keys % P, h].double()
            Q = s["q"][rows, h * G:(h + 1) * G].double()
            x = torch.einsum("tgd,kd->tgk", Q, K) * s["scale"]
            x.masked_fill_(hidden[:, None], -math.inf)
            z = torch.logsumexp(x, -1)
            lse[rows, h * G:(h + 1) * G] = z
            out[rows, h * G:(h + 1) * G] = torch.einsum("tgk,kd->tgd", (x - z[..., None]).exp(), V)
        start += n
    return {"out": out, "lse": lse}


def _exact_keep(c, s):
    """The bookkeeping, row by row on the host (the caches' bytes have no other form)."""
    P = c["page"]
    refs, table, lens = s["refs"].tolist(), s["table"].tolist(), s["lens"].tolist()
    for b, (before, d, kept) in enumerate(_accepted(c)):
        length = before + len(kept)
        for j in range(-(-length // P), -(-(before + d) // P)):
            refs[table[b][j]] -= 1
            table[b][j] = -1
        lens[b] = length
    as_int = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return {"caches": None, "refs": as_int(refs), "lens": as_int(lens), "table": as_int(table)}
