"""Measured cases of normed rotary append, windowed attention and the pages of a cache.

Five operators of a serving loop over a paged key/value cache:

* ``norm``     root-mean-square norms of the new tokens' query and key heads,
  rotary positions, and the append of keys and values, in one pass;
* ``window``   causal attention of new tokens (one, or a prompt's) that see the
  last tokens up to a window and a few first ones;
* ``pages``    page tables kept to the pages that the sequences need: the others
  given back, missing ones taken from the free ones;
* ``fork``     children of sequences: whole pages shared, a partly filled last
  page copied;
* ``compact``  the accepted ones of a sequence's drafted tokens moved to the front.

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is set, through the package's entry points. ``exact`` computes them in
64 bits from the definition, one sequence at a time.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ALL = 2 ** 31 - 1   # a window that hides nothing
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    H = {"Hq": 48, "Hkv": 8, "D": 128}   # 48 heads of 128: a model width of 6144
    return [
        # one new token of one sequence: launch latency is all there is
        dict(name="norm_1_token", op="norm", B=1, T=1, ctx=5000, page=64, rot=128, half=True, src="bf16",
             dtype="bf16", wtype="fp32", **H),
        # a chunk of four long prompts going into the cache
        dict(name="norm_prefill_16k", op="norm", B=4, T=4093, ctx=1000, page=64, rot=128, half=True, src="bf16",
             dtype="bf16", wtype="bf16", **H),
        # one token of a long chat: the window is all it reads
        dict(name="window_1_token", op="window", B=1, T=1, ctx=20011, page=64, W=4096, S=4, dtype="bf16",
             out="bf16", **H),
        # a decode batch of long chats
        dict(name="window_decode_64", op="window", B=64, T=1, ctx=30011, page=64, W=4096, S=4, dtype="bf16",
             out="bf16", Hq=32, Hkv=8, D=128),
        # long prompts, every token with its own window
        dict(name="window_prefill_12k", op="window", B=3, T=4093, ctx=2000, page=64, W=2048, S=4, dtype="bf16",
             out="bf16", **H),
        # ragged chunks, an odd window and first tokens that end inside a page, narrow heads, five
        # queries a head, small pages, fp32 outputs
        dict(name="window_chunks_fp32", op="window", B=16, T=301, ctx=6000, page=16, W=513, S=17, dtype="fp16",
             out="fp32", Hq=40, Hkv=8, D=64),
        # a decode batch's step: windows that move on, pages for the next drafts
        dict(name="pages_step_64", op="pages", B=64, ctx=30011, page=64, W=4096, S=4, more=8, ended=0),
        # a large batch without windows, a quarter of its sequences over, prompts coming in
        dict(name="pages_batch_1024", op="pages", B=1024, ctx=12007, page=16, W=ALL, S=0, more=1500, ended=4),
        # four continuations of one chat
        dict(name="fork_4", op="fork", B=1, F=4, ctx=5003, page=64, dtype="bf16", Hkv=8, D=128),
        # a beam's reordering: 256 sequences of 64 parents, half a page each to copy
        dict(name="fork_256", op="fork", B=64, F=256, ctx=9001, page=128, dtype="bf16", Hkv=8, D=128),
        # a tree's accepted path
        dict(name="compact_1_tree", op="compact", B=1, T=16, ctx=777, page=64, dtype="bf16", Hkv=8, D=128),
        # trees of a batch, and the sums beside their keys
        dict(name="compact_256_trees", op="compact", B=256, T=61, ctx=1500, page=32, dtype="fp16", Hkv=8, D=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "window", "window", "window", "pages", "fork", "compact"])
    D, Hkv, G = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    c = dict(op=op, page=page)
    if op == "pages":
        c.update(B=_log(rng, 1, 1000), ctx=_log(rng, 10, 30000), W=rng.choice([ALL, _log(rng, 1, 8000)]),
                 S=rng.choice([0, 4, 17, 130]), more=_log(rng, 1, 1500), ended=rng.choice([0, 2, 4, 7]))
        c["ctx"] = max(1, min(c["ctx"], 700000 * page // c["B"]))
        return c
    c.update(dtype=rng.choice(["bf16", "fp16"]), Hkv=Hkv, D=D)
    if op == "norm":
        c.update(B=_log(rng, 1, 64), Hq=G * Hkv, ctx=_log(rng, 1, 80000), rot=rng.choice([D, D // 2, D // 4]),
                 half=rng.random() < 0.6, src=rng.choice([c["dtype"], "fp32"]),
                 wtype=rng.choice([c["dtype"], "fp32"]))
        # within the largest listed case's bytes
        row = (c["Hq"] + 2 * Hkv) * D * (6 if c["src"] == "fp32" else 4)
        c["T"] = max(1, min(_log(rng, 1, 4096), 480000000 // row // c["B"]))
        c["ctx"] = min(c["ctx"], 1200000 // c["B"])
        return c
    if op == "window":
        T = rng.choice([1, _log(rng, 2, 40), _log(rng, 40, 4096)])
        c.update(Hq=G * Hkv, T=T, W=rng.choice([ALL, _log(rng, 1, 8000), _log(rng, 100, 8000)]),
                 S=rng.choice([0, 4, 17, 130]), out=rng.choice([c["dtype"], c["dtype"], "fp32"]))
        # within the largest listed case's keys and scores
        most = min(380000 * 1024 // (Hkv * D), 3000000000 // (T * G * Hkv))
        c["ctx"] = _log(rng, 1, 100000)
        c["B"] = max(1, min(_log(rng, 1, 64), most // (c["ctx"] + T)))
        c["ctx"] = max(1, min(c["ctx"], most // c["B"] - T))
        return c
    if op == "fork":
        c.update(B=_log(rng, 1, 64), F=_log(rng, 1, 256), ctx=_log(rng, 1, 9000))
        return c
    c.update(B=_log(rng, 1, 256), T=_log(rng, 2, 200), ctx=_log(rng, 1, 1500))
    c["B"] = max(1, min(c["B"], 15600 // c["T"]))
    return c


# ------------------------------------------------------------------ shapes that the case alone sets

def _contexts(c):
    """Cached tokens of each sequence before the call: ragged, the first the longest."""
    n, B = c["ctx"], c["B"]
    return [n - (b * (n // 2)) // max(B, 1) - (b * 37) % max(n // 16, 1) for b in range(B)]


def _drafts(c):
    """New tokens of each sequence (ragged where there are several)."""
    T = c["T"]
    return [max(1, T - (b % 3) * (T // 8)) for b in range(c["B"])]


def _pairs(ctx, T, W, S):
    """(token, seen slot) pairs of T new tokens after ctx, and the slots that some token sees."""
    p = np.arange(ctx, ctx + T, dtype=np.int64)
    near = np.minimum(p + 1, W)
    first = np.minimum(S, p + 1 - near)
    return int((near + first).sum()), int(T + near[0] - 1 + first[-1])


def work(c):
    page = c["page"]
    if c["op"] == "norm":
        D, n = c["D"], sum(_drafts(c))
        e = 4 if c["src"] == "fp32" else 2
        heads = c["Hq"] + c["Hkv"]
        return {"bytes": n * (heads + c["Hkv"]) * D * (e + 2), "flops": n * heads * (3 * c["rot"] + 4 * D)}
    if c["op"] == "window":
        D, Hkv, n = c["D"], c["Hkv"], sum(_drafts(c))
        seen = [_pairs(a, t, c["W"], c["S"]) for a, t in zip(_contexts(c), _drafts(c))]
        by = sum(k for _, k in seen) * Hkv * D * 4 + n * c["Hq"] * (D * (2 + (4 if c["out"] == "fp32" else 2)) + 4)
        return {"bytes": by, "flops": 4 * D * c["Hq"] * sum(k for k, _ in seen)}
    if c["op"] == "pages":
        width, _ = _page_sizes(c)
        return {"bytes": 4 * c["B"] * (width + 2), "flops": 0}
    if c["op"] == "fork":
        lens = _contexts(c)
        rows = sum(lens[_parent(i, c)] % page for i in range(c["F"]))
        width = -(-max(lens) // page)
        return {"bytes": rows * c["Hkv"] * c["D"] * 8 + 8 * c["F"] * width, "flops": 0}
    moved = sum(max(0, len(k) - _still(k)) for k in _paths(c))
    return {"bytes": moved * c["Hkv"] * (8 * c["D"] + 8) + 8 * c["B"], "flops": 0}


def _page_sizes(c):
    """A table's width and the pool's pages of a ``pages`` case."""
    width = -(-(c["ctx"] + c["more"]) // c["page"])
    held = sum(-(-n // c["page"]) for n in _contexts(c))
    return width, held + c["B"] * (-(-c["more"] // c["page"]) + 1)


def _parent(i, c):
    return (i * 7) % c["B"]


def _paths(c):
    """Accepted drafts of each sequence: ascending indices (of a path through its tree)."""
    rng = np.random.default_rng(c["B"] * 1000 + c["T"])
    got = []
    for t in _drafts(c):
        n = int(rng.integers(1, min(t, 8) + 1))
        got.append(np.sort(rng.choice(t, n, replace=False)))
    return got


def _still(keep):
    """How many tokens of a path are in their places already."""
    return int((np.asarray(keep) == np.arange(len(keep))).sum())


# ------------------------------------------------------------------ inputs

def _needed(c, lens, more, width):
    """Which pages of each sequence are needed: [B][width]."""
    first = np.arange(width, dtype=np.int64) * c["page"]
    lens, more = np.asarray(lens, np.int64)[:, None], np.asarray(more, np.int64)[:, None]
    return (first < lens + more) & ((first < c["S"]) | (first + c["page"] > lens - c["W"] + 1))


def _tables(held, g, dev):
    """Page tables (-1: none) over a shuffled pool for the pages held [B][width], and the pages."""
    pages = int(held.sum())
    order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32).cpu().numpy()
    table = np.full(held.shape, -1, np.int32)
    table[held] = order
    return table, pages


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    page, ctx = c["page"], _contexts(c)

    def normal(*shape, dtype=None, scale=1.0, mean=0.0):
        x = torch.empty(shape, dtype=dtype or DTYPES[c["dtype"]], device=dev)
        return x.normal_(mean, scale, generator=g)

    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(dev)  # noqa: E731
    s = {"case": c}
    if c["op"] == "pages":
        # what the tables held for shorter lengths; some sequences are over by now
        width, pages = _page_sizes(c)
        step = rng.integers(0, 3 * page, c["B"])
        before = np.maximum(0, np.array(ctx) - step)
        table, held = _tables(_needed(c, before, step * 0 + page, width), g, dev)
        pages = max(pages, held)
        spread = np.sort(rng.choice(pages, held, replace=False)).astype(np.int32)
        table[table >= 0] = spread[table[table >= 0]]
        refs = np.zeros(pages, np.int32)
        refs[table[table >= 0]] = 1
        over = (np.arange(c["B"]) % c["ended"] == 1) if c["ended"] else np.zeros(c["B"], bool)
        s["table0"], s["refs0"] = i32(table), i32(refs)
        s["table"], s["refs"] = s["table0"].clone(), s["refs0"].clone()
        s["lens"] = i32(np.where(over, 0, ctx))
        s["more"] = i32(np.where(over, 0, rng.integers(1, c["more"] + 1, c["B"])))
        return s
    if c["op"] == "fork":
        lens, F, B = np.array(ctx), c["F"], c["B"]
        # sequences that share their first pages, as children of one prompt do
        width = -(-max(ctx) // page)
        held = np.arange(width) * page < lens[:, None]
        common = min(ctx) // page // 2
        held[1:, :common] = False
        table, n = _tables(held, g, dev)
        table[1:, :common] = table[0, :common]
        pages = n + F + 3
        spread = np.sort(rng.choice(pages, n, replace=False)).astype(np.int32)
        table[table >= 0] = spread[table[table >= 0]]
        s["table"], s["refs0"] = i32(table), i32(np.bincount(table[table >= 0], minlength=pages))
        s["refs"] = s["refs0"].clone()
        s["lens"], s["parent"] = i32(lens), i32([_parent(i, c) for i in range(F)])
        s["k"], s["v"] = normal(pages, c["Hkv"], page, c["D"]), normal(pages, c["Hkv"], page, c["D"])
        return s
    drafts = _drafts(c)
    n = sum(drafts)
    D, Hkv = c["D"], c["Hkv"]
    s["ctx"], s["cu"] = i32(ctx), i32([0] + list(np.cumsum(drafts)))
    total = [a + t for a, t in zip(ctx, drafts)]
    held = np.arange(-(-max(total) // page)) * page < np.array(total)[:, None]
    if c["op"] == "window":
        held &= _needed(c, ctx, drafts, held.shape[1])   # what lies behind the windows has been given back
    table, pages = _tables(held, g, dev)
    s["table"] = i32(table)
    s["k"], s["v"] = normal(pages, Hkv, page, D), normal(pages, Hkv, page, D)
    if c["op"] == "norm":
        # the projections' output: the heads of q, k and v side by side in each token's row
        s["qkv"] = normal(n, c["Hq"] + 2 * Hkv, D, dtype=DTYPES[c["src"]], scale=3.0)
        s["wq"], s["wk"] = (normal(D, dtype=DTYPES[c["wtype"]], scale=0.25, mean=1.0) for _ in range(2))
        s["pos"] = i32(np.concatenate([np.arange(a, b) for a, b in zip(ctx, total)]))
        i = np.arange(c["rot"] // 2, dtype=np.float64)
        s["inv_freq"] = torch.from_numpy(10000.0 ** (-2.0 * i / c["rot"])).to(dev)
    elif c["op"] == "window":
        s["q"] = normal(n, c["Hq"], D, scale=2.0)   # scores of standard deviation 2: some keys stand out
    else:
        keep = np.zeros(n, np.int32)
        for first, path in zip(np.cumsum([0] + drafts), _paths(c)):
            keep[first:first + len(path)] = path
        s["keep"], s["kept"] = i32(keep), i32([len(p) for p in _paths(c)])
        s["acc"] = torch.empty(pages, Hkv, page, device=dev).uniform_(0.0, 1.0, generator=g)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        return _RUN_OWN[c["op"]](s, c)
    return _RUN_PLAIN[c["op"]](s, c)


def _slots(s, c):
    """Page and row in the cache of every new token."""
    n = s["pos"].shape[0]
    tok = torch.arange(n, device=s["cu"].device)
    b = torch.searchsorted(s["cu"].long(), tok, right=True) - 1
    slot = s["ctx"].long()[b] + tok - s["cu"].long()[b]
    return s["table"].long()[b, slot // c["page"]], slot % c["page"]


def _rotate(x, cos, sin, rot, half):
    r, rest = x[..., :rot], x[..., rot:]
    if half:
        a, b = r[..., : rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, rest], -1)


def _normed(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _plain_norm(s, c):
    Hq, Hkv = c["Hq"], c["Hkv"]
    q, k, v = s["qkv"].split([Hq, Hkv, Hkv], 1)
    angle = s["pos"].double()[:, None, None] * s["inv_freq"]      # far positions need 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    page, row = _slots(s, c)
    s["k"][page, :, row] = _rotate(_normed(k, s["wk"]), cos, sin, c["rot"], c["half"]).to(s["k"].dtype)
    s["v"][page, :, row] = v.float().to(s["v"].dtype)
    q = _rotate(_normed(q, s["wq"]), cos, sin, c["rot"], c["half"])
    return {"q": q.to(s["k"].dtype), "k": s["k"], "v": s["v"]}


def _plain_window(s, c):
    dev, (B, T, Hkv, D, W, S) = s["q"].device, (c["B"], c["T"], c["Hkv"], c["D"], c["W"], c["S"])
    G = c["Hq"] // Hkv
    cu, ctx, table = s["cu"].long(), s["ctx"].long(), s["table"].long()
    new = cu[1:] - cu[:-1]
    # the slots that can be seen: the first ones, and those from the first window's start on
    L = table.shape[1] * c["page"]
    span = min(L, W + T - 1)
    start = (ctx + new - span).clamp(min=0)
    first = torch.arange(min(S, L), device=dev).expand(B, -1)
    slot = torch.cat([first, start[:, None] + torch.arange(span, device=dev)], 1)
    there = torch.cat([first < start[:, None], torch.ones(B, span, dtype=torch.bool, device=dev)], 1)
    there &= slot < (ctx + new)[:, None]
    slot = torch.where(there, slot, 0)
    page = table.gather(1, slot // c["page"])
    page = torch.where(page >= 0, page, 0)
    # queries by sequence, padded to T; keys and values by sequence
    j = torch.arange(T, device=dev)
    live = j < new[:, None]
    at = torch.where(live, cu[:-1, None] + j, 0)
    qf = s["q"].float()[at].view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    kf = s["k"][page, :, slot % c["page"]].float().permute(0, 2, 1, 3)
    n = slot.shape[1]
    x = torch.matmul(qf, kf.transpose(2, 3)).view(B, Hkv, T, G, n) * (1.0 / math.sqrt(D))
    del kf
    p = (ctx[:, None] + j)[:, :, None]
    seen = there[:, None] & (slot[:, None] <= p) & ((slot[:, None] > p - W) | (slot[:, None] < S))
    x = torch.where(seen[:, None, :, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    w = torch.exp(x - top)
    del x
    z = w.sum(-1, keepdim=True)
    vf = s["v"][page, :, slot % c["page"]].float().permute(0, 2, 1, 3)
    vf = torch.where(there[:, None, :, None], vf, 0.0)
    o = torch.matmul(w.view(B, Hkv, T * G, n), vf).view(B, Hkv, T, G, D) / torch.where(z == 0, 1.0, z)
    lse = (top + z.log())[..., 0].permute(0, 2, 1, 3)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, c["Hq"], D)[live]
    return {"o": o.to(DTYPES[c["out"]]), "lse": lse.reshape(B, T, c["Hq"])[live]}


def _plain_pages(s, c):
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    table, refs, page = s["table"], s["refs"], c["page"]
    first = torch.arange(table.shape[1], device=table.device) * page
    lens, end = s["lens"].long()[:, None], (s["lens"] + s["more"]).long()[:, None]
    need = (first < end) & ((first < c["S"]) | (first + page > lens - c["W"] + 1))
    back = (table >= 0) & ~need
    refs.index_add_(0, table[back], torch.full((1,), -1, dtype=torch.int32, device=table.device).expand(int(back.sum())))
    table.masked_fill_(back, -1)
    at = torch.nonzero(need & (table < 0))                        # in order of sequence and page
    free = torch.nonzero(refs == 0)[: at.shape[0], 0].int()       # the lowest first
    at = at[: free.shape[0]]
    table[at[:, 0], at[:, 1]] = free
    refs[free.long()] = 1
    return {"table": table, "refs": refs}


def _plain_fork(s, c):
    s["refs"].copy_(s["refs0"])
    refs, page = s["refs"], c["page"]
    rows, lens = s["table"][s["parent"].long()], s["lens"][s["parent"].long()]
    first = torch.arange(rows.shape[1], device=rows.device) * page
    whole = (first + page <= lens[:, None]) & (rows >= 0)
    part = (first < lens[:, None]) & (first + page > lens[:, None]) & (rows >= 0)
    table = torch.where(whole, rows, -1)
    refs.add_(torch.bincount(rows[whole], minlength=refs.shape[0]).int())
    at = torch.nonzero(part)
    free = torch.nonzero(refs == 0)[: at.shape[0], 0].int()
    at = at[: free.shape[0]]
    table[at[:, 0], at[:, 1]] = free
    refs[free.long()] = 1
    moves = torch.full((rows.shape[0], 3), -1, dtype=torch.int32, device=rows.device)
    moves[:, 2] = 0
    n = lens[at[:, 0]] % page
    moves[at[:, 0]] = torch.stack([rows[at[:, 0], at[:, 1]], free, n], 1)
    i, r = torch.nonzero(torch.arange(page, device=rows.device) < moves[:, 2:], as_tuple=True)
    src, dst = moves[i, 0].long(), moves[i, 1].long()
    s["k"][dst, :, r] = s["k"][src, :, r]
    s["v"][dst, :, r] = s["v"][src, :, r]
    return {"table": table, "lens": lens, "moves": moves, "refs": refs, "k": s["k"], "v": s["v"]}


def _plain_compact(s, c):
    cu, ctx, page = s["cu"].long(), s["ctx"].long(), c["page"]
    tok = torch.arange(s["keep"].shape[0], device=cu.device)
    b = torch.searchsorted(cu, tok, right=True) - 1
    i = tok - cu[b]
    b, i, d = (x[i < s["kept"].long()[b]] for x in (b, i, s["keep"].long()))
    src, dst = ctx[b] + d, ctx[b] + i
    sp, dp = s["table"].long()[b, src // page], s["table"].long()[b, dst // page]
    s["k"][dp, :, dst % page] = s["k"][sp, :, src % page]
    s["v"][dp, :, dst % page] = s["v"][sp, :, src % page]
    s["acc"][dp, :, dst % page] = s["acc"][sp, :, src % page]
    return {"ctx": s["ctx"] + s["kept"], "k": s["k"], "v": s["v"], "acc": s["acc"]}


def _cache(s):
    import int4_group_quantized_gs64_gb300 as qmv
    if "cache" not in s:
        s["cache"] = qmv.AttnCache(s["k"], s["v"])
    return qmv, s["cache"]


def _own_norm(s, c):
    qmv, cache = _cache(s)
    Hq, Hkv = c["Hq"], c["Hkv"]
    q, k, v = s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv], s["qkv"][:, Hq + Hkv:]
    out = qmv.attn_norm_rope_append(cache, q, k, v, s["wq"], s["wk"], s["pos"], s["inv_freq"], s["table"], s["ctx"],
                                    s["cu"], eps=EPS, interleaved=not c["half"])
    return {"q": out, "k": s["k"], "v": s["v"]}


def _own_window(s, c):
    qmv, cache = _cache(s)
    if "ws" not in s:
        n = qmv.attn_window_workspace_bytes(cache, c["Hq"], c["B"], s["q"].shape[0], c["T"], s["table"].shape[1])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=s["k"].device)
    o, lse = qmv.attn_window(cache, s["q"], s["table"], s["ctx"], s["cu"], c["T"], window=c["W"], sinks=c["S"],
                             o_dtype=DTYPES[c["out"]], ws=s["ws"])
    return {"o": o, "lse": lse}


def _own_pages(s, c):
    import int4_group_quantized_gs64_gb300 as qmv
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    qmv.attn_pages_update(s["refs"], s["table"], s["lens"], s["more"], c["page"], window=c["W"], sinks=c["S"])
    return {"table": s["table"], "refs": s["refs"]}


def _own_fork(s, c):
    qmv, cache = _cache(s)
    s["refs"].copy_(s["refs0"])
    table, lens, moves = qmv.attn_pages_fork(s["refs"], s["table"], s["lens"], s["parent"], c["page"])
    qmv.attn_pages_copy(cache, cache, moves)
    return {"table": table, "lens": lens, "moves": moves, "refs": s["refs"], "k": s["k"], "v": s["v"]}


def _own_compact(s, c):
    qmv, cache = _cache(s)
    ctx = qmv.attn_compact(cache, s["table"], s["ctx"], s["cu"], s["keep"], s["kept"], acc=s["acc"])
    return {"ctx": ctx, "k": s["k"], "v": s["v"], "acc": s["acc"]}


_RUN_PLAIN = {"norm": _plain_norm, "window": _plain_window, "pages": _plain_pages, "fork": _plain_fork,
              "compact": _plain_compact}
_RUN_OWN = {"norm": _own_norm, "window": _own_window, "pages": _own_pages, "fork": _own_fork,
            "compact": _own_compact}


# ------------------------------------------------------------------ in 64 bits, one sequence at a time

def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "window": _exact_window, "pages": _exact_pages, "fork": _exact_fork,
            "compact": _exact_compact}[c["op"]](s, c)


def _exact_norm(s, c):
    Hq, Hkv, rot, D = c["Hq"], c["Hkv"], c["rot"], c["D"]
    k, v = s["k"].double(), s["v"].double()
    x = s["qkv"].double()
    for part, w in ((slice(0, Hq), s["wq"]), (slice(Hq, Hq + Hkv), s["wk"])):
        length = torch.linalg.vector_norm(x[:, part], dim=-1, keepdim=True)
        x[:, part] *= w.double() / torch.sqrt(length * length / D + EPS)
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=x.device),
                       torch.outer(s["pos"].double(), s["inv_freq"]))           # [N][rot/2], complex
    pairs = x[:, :Hq + Hkv, :rot]
    if c["half"]:
        z = torch.complex(pairs[..., : rot // 2].contiguous(), pairs[..., rot // 2:].contiguous()) * turn[:, None]
        x[:, :Hq + Hkv, :rot] = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(pairs.reshape(*pairs.shape[:2], rot // 2, 2).contiguous()) * turn[:, None]
        x[:, :Hq + Hkv, :rot] = torch.view_as_real(z).reshape(pairs.shape)
    cu, ctx, table = s["cu"].tolist(), s["ctx"].tolist(), s["table"].cpu().numpy()
    for b in range(c["B"]):
        slot = ctx[b] + np.arange(cu[b + 1] - cu[b])
        page = torch.from_numpy(table[b, slot // c["page"]]).long().to(x.device)
        row = torch.from_numpy(slot % c["page"]).to(x.device)
        k[page, :, row] = x[cu[b]:cu[b + 1], Hq:Hq + Hkv]
        v[page, :, row] = x[cu[b]:cu[b + 1], Hq + Hkv:]
    return {"q": x[:, :Hq].contiguous(), "k": k, "v": v}


def _exact_window(s, c):
    D, Hkv, page = c["D"], c["Hkv"], c["page"]
    G, dev = c["Hq"] // Hkv, s["q"].device
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=dev)
    for b in range(c["B"]):
        t, n = cu[b + 1] - cu[b], ctx[b] + cu[b + 1] - cu[b]
        j = torch.cat([torch.arange(min(c["S"], max(0, ctx[b] - c["W"] + 1))),
                       torch.arange(max(0, ctx[b] - c["W"] + 1), n)]).to(dev)
        back = torch.arange(ctx[b], n, device=dev)[:, None] - j     # how far back a slot lies
        see = (back >= 0) & ((back < c["W"]) | (j < c["S"]))
        at = s["table"][b].long()[j // page]
        for h in range(Hkv):
            k, v = s["k"][at, h, j % page].double(), s["v"][at, h, j % page].double()
            for g in range(G):
                x = s["q"][cu[b]:cu[b + 1], h * G + g].double() @ k.T / math.sqrt(D)
                x.masked_fill_(~see, -math.inf)
                e = torch.logsumexp(x, 1)
                o[cu[b]:cu[b + 1], h * G + g] = x.sub_(e[:, None]).exp_() @ v
                lse[cu[b]:cu[b + 1], h * G + g] = e
    return {"o": o, "lse": lse}


def _exact_pages(s, c):
    table, refs = s["table0"].cpu().numpy().copy(), s["refs0"].cpu().numpy().copy()
    lens, more = s["lens"].tolist(), s["more"].tolist()
    need = _needed(c, lens, more, table.shape[1])
    for b in range(c["B"]):
        for i in np.flatnonzero((table[b] >= 0) & ~need[b]):
            refs[table[b, i]] -= 1
            table[b, i] = -1
    free = list(np.flatnonzero(refs == 0)[::-1])
    for b in range(c["B"]):
        for i in np.flatnonzero((table[b] < 0) & need[b]):
            if free:
                table[b, i] = free.pop()
                refs[table[b, i]] = 1
    return {"table": torch.from_numpy(table), "refs": torch.from_numpy(refs)}


def _exact_fork(s, c):
    table, refs = s["table"].cpu().numpy(), s["refs0"].cpu().numpy().copy()
    lens, parent, page = s["lens"].tolist(), s["parent"].tolist(), c["page"]
    k, v = s["k"].double(), s["v"].double()
    new, moves = np.full((c["F"], table.shape[1]), -1, np.int32), np.zeros((c["F"], 3), np.int32)
    moves[:, :2] = -1
    for i, p in enumerate(parent):
        n = lens[p] // page
        new[i, :n] = table[p, :n]
        np.add.at(refs, table[p, :n][table[p, :n] >= 0], 1)
    free = list(np.flatnonzero(refs == 0)[::-1])
    for i, p in enumerate(parent):
        n, rows = divmod(lens[p], page)
        if rows and free:
            new[i, n] = free.pop()
            refs[new[i, n]] = 1
            moves[i] = table[p, n], new[i, n], rows
            k[int(new[i, n]), :, :rows] = k[int(table[p, n]), :, :rows]
            v[int(new[i, n]), :, :rows] = v[int(table[p, n]), :, :rows]
    return {"table": torch.from_numpy(new), "lens": torch.tensor([lens[p] for p in parent], dtype=torch.int32),
            "moves": torch.from_numpy(moves), "refs": torch.from_numpy(refs), "k": k, "v": v}


def _exact_compact(s, c):
    k, v, acc = s["k"].double(), s["v"].double(), s["acc"].double()
    ctx, table, page = s["ctx"].tolist(), s["table"].cpu().numpy(), c["page"]
    for b, path in enumerate(_paths(c)):
        src, dst = ctx[b] + path, ctx[b] + np.arange(len(path))
        sp, sr, dp, dr = (torch.from_numpy(x.astype(np.int64)).to(k.device) for x in
                          (table[b, src // page], src % page, table[b, dst // page], dst % page))
        for pool in (k, v, acc):
            pool[dp, :, dr] = pool[sp, :, sr].clone()
    kept = [len(p) for p in _paths(c)]
    return {"ctx": torch.tensor([a + n for a, n in zip(ctx, kept)], dtype=torch.int32), "k": k, "v": v, "acc": acc}
