"""Measured cases of the attention operators over a paged key/value cache.

Three operators that a decode or speculative-decoding step runs around the
expert layers:

* ``rope``   rotary positions of the new tokens' queries and keys, and the
  append of the rotated keys and the values to the paged cache;
* ``tree``   attention of every sequence's drafted tokens (a tree, or one
  token) over its cached tokens and over the drafted tokens the tree allows,
  optionally adding each cached token's attention weight to its running sum;
* ``evict``  the cached tokens with the largest running sums (with the first
  and the most recent ones) kept, in order, in fresh pages.

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is set, through the package's entry points. ``exact`` computes them in
64 bits from the definition, one sequence at a time.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    H = {"Hq": 48, "Hkv": 8, "D": 128}   # 48 heads of 128: a model width of 6144
    return [
        # one new token of one sequence: launch latency is all there is
        dict(name="rope_1_token", op="rope", B=1, T=1, ctx=5000, page=64, rot=128, half=True,
             src="bf16", dtype="bf16", base=10000.0, stretch=1.0, **H),
        # drafted trees of 16 sequences from the fp32 projections: interleaved
        # pairs, half of each head rotated, positions stretched for long contexts
        dict(name="rope_trees_fp32", op="rope", B=16, T=33, ctx=70001, page=16, rot=64, half=False,
             src="fp32", dtype="fp16", base=500000.0, stretch=8.0, Hq=32, Hkv=8, D=128),
        # a chunk of four long prompts going into the cache
        dict(name="rope_prefill_16k", op="rope", B=4, T=4093, ctx=1000, page=64, rot=128, half=True,
             src="bf16", dtype="bf16", base=10000.0, stretch=1.0, **H),
        # one sequence, one token, a short context: the latency of a chat's start
        dict(name="tree_1_token_short", op="tree", B=1, T=1, ctx=777, page=64, dtype="bf16",
             out="bf16", acc=False, **H),
        # a full decode batch, ragged contexts
        dict(name="tree_decode_64", op="tree", B=64, T=1, ctx=8191, page=64, dtype="bf16",
             out="bf16", acc=False, Hq=32, Hkv=8, D=128),
        # one very long context, a single token, outputs for the fp32 projections
        dict(name="tree_1_token_200k", op="tree", B=1, T=1, ctx=200003, page=128, dtype="fp16",
             out="fp32", acc=False, **H),
        # drafted trees of 64 nodes: 512 query rows per key/value head
        dict(name="tree_64_nodes", op="tree", B=8, T=64, ctx=8200, page=64, dtype="bf16",
             out="bf16", acc=False, Hq=64, Hkv=8, D=128),
        # a decode batch that also keeps the running attention weights
        dict(name="tree_decode_weights", op="tree", B=32, T=1, ctx=10007, page=32, dtype="bf16",
             out="bf16", acc=True, **H),
        # odd trees, narrow heads, five queries a head, small pages, running weights
        dict(name="tree_21_nodes_weights", op="tree", B=16, T=21, ctx=6000, page=16, dtype="fp16",
             out="fp16", acc=True, Hq=40, Hkv=8, D=64),
        # a chat's cache cut to a quarter
        dict(name="evict_4k_to_1k", op="evict", B=1, ctx=4099, page=64, budget=1024, sink=4,
             recent=128, dtype="bf16", Hkv=8, D=128),
        # a ragged batch, some of it below the budget
        dict(name="evict_batch_16k", op="evict", B=16, ctx=16411, page=64, budget=4096, sink=4,
             recent=257, dtype="bf16", Hkv=8, D=128),
        # very long contexts cut hard
        dict(name="evict_300k", op="evict", B=2, ctx=300007, page=128, budget=16384, sink=16,
             recent=1024, dtype="fp16", Hkv=8, D=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    return {k: 3071 if v == 3072 else v for k, v in _draw(rng).items()}   # that size is left out


def _draw(rng):
    op = rng.choice(["rope", "tree", "tree", "evict"])
    D, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    G = 5 if G * Hkv * D == 3072 else G
    c = dict(op=op, page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "fp16"]), Hkv=Hkv, D=D)
    if op == "rope":
        c.update(B=_log(rng, 1, 64), Hq=G * Hkv, ctx=_log(rng, 1, 80000), rot=rng.choice([D, D // 2, D // 4]),
                 half=rng.random() < 0.6, src=rng.choice([c["dtype"], "fp32"]),
                 base=rng.choice([10000.0, 500000.0]), stretch=rng.choice([1.0, 4.0, 8.0]))
        # within the largest listed case's bytes
        row = (c["Hq"] + 2 * Hkv) * D * (6 if c["src"] == "fp32" else 4)
        c["T"] = max(1, min(_log(rng, 1, 4096), 480000000 // row // c["B"]))
        c["ctx"] = min(c["ctx"], 1200000 // c["B"])
        return c
    c["ctx"] = _log(rng, 40, 200000)
    if op == "tree":
        T = rng.choice([1, 1, _log(rng, 2, 100)])
        c.update(Hq=G * Hkv, T=T, out=rng.choice([c["dtype"], c["dtype"], "fp32"]), acc=rng.random() < 0.4)
        # within the largest listed case's keys, products and scores
        most = min(380000 * 1024 // (Hkv * D), int(0.94e11) // (4 * T * G * Hkv * D), 260000000 // (T * G * Hkv))
        c["B"] = max(1, min(_log(rng, 1, 64), most // (c["ctx"] + T)))
        c["ctx"] = max(1, min(c["ctx"], most // c["B"] - T))
        return c
    c["B"] = max(1, min(_log(rng, 1, 32), 600000 // c["ctx"]))
    c["budget"] = max(24, min(_log(rng, c["ctx"] // 32 + 1, c["ctx"]), 63000 * 1024 // (c["B"] * Hkv * D)))
    c["sink"] = rng.choice([0, 4, 16])
    c["recent"] = rng.randrange(0, c["budget"] - c["sink"] + 1) // 2
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


def work(c):
    D, Hkv = c["D"], c["Hkv"]
    if c["op"] == "rope":
        n = sum(_drafts(c))
        e = 4 if c["src"] == "fp32" else 2
        return {"bytes": n * (c["Hq"] + 2 * Hkv) * D * (e + 2), "flops": n * (c["Hq"] + Hkv) * c["rot"] * 3}
    if c["op"] == "tree":
        keys = [a + t for a, t in zip(_contexts(c), _drafts(c))]
        n = sum(_drafts(c))
        by = sum(keys) * Hkv * D * 4 + n * c["Hq"] * D * (2 + (4 if c["out"] == "fp32" else 2)) + n * c["Hq"] * 4
        if c["acc"]:
            by += sum(keys) * Hkv * 8
        return {"bytes": by, "flops": sum(4 * k * t * c["Hq"] * D for k, t in zip(keys, _drafts(c)))}
    lens = _contexts(c)
    kept = sum(min(n, c["budget"]) for n in lens)
    return {"bytes": Hkv * (4 * sum(n for n in lens if n > c["budget"]) + kept * (2 * D * 2 * 2 + 8 + 4)), "flops": 0}


# ------------------------------------------------------------------ inputs

def _pool(c, lens, g, dev):
    """Page table of sequences of `lens` tokens over a shuffled pool, and the pool's pages."""
    page = c["page"]
    need = [-(-n // page) for n in lens]
    width, pages = max(need), sum(need)
    order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32).cpu().numpy()
    table = np.zeros((len(lens), width), np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table).to(dev), pages


def _trees(drafts, rng):
    """A random tree over each sequence's drafts: bit j of a token's words is set for itself and its ancestors."""
    W = -(-max(drafts) // 32)
    rows = []
    for t in drafts:
        bits = []
        for j in range(t):
            p = -1 if j == 0 else int(rng.integers(max(0, j - 8), j))
            bits.append((bits[p] if p >= 0 else 0) | (1 << j))
        rows += [[(v >> (32 * w)) & 0xFFFFFFFF for w in range(W)] for v in bits]
    return np.array(rows, np.uint32).view(np.int32)


def _depths(mask):
    return np.unpackbits(mask.view(np.uint8), axis=1).sum(1).astype(np.int32) - 1


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt, D, Hkv, page = DTYPES[c["dtype"]], c["D"], c["Hkv"], c["page"]

    def normal(*shape, dtype=dt, scale=1.0):
        x = torch.empty(shape, dtype=dtype, device=dev)
        return x.normal_(0.0, scale, generator=g)

    s = {"case": c}
    ctx = _contexts(c)
    if c["op"] == "evict":
        s["table"], pages = _pool(c, ctx, g, dev)
        s["lens"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
        s["k"], s["v"] = normal(pages, Hkv, page, D), normal(pages, Hkv, page, D)
        # heavy-tailed sums of attention weights; about a tenth never attended to, and so tied at zero
        a = torch.empty(pages, Hkv, page, device=dev).normal_(0.0, 2.0, generator=g).exp_()
        a.mul_(torch.empty_like(a).uniform_(0.0, 1.0, generator=g).gt_(0.1))
        s["acc"] = a
        s["dst_table"], dpages = _pool(c, [min(c["budget"], max(ctx))] * c["B"], g, dev)
        s["dst_k"] = torch.zeros(dpages, Hkv, page, D, dtype=dt, device=dev)
        s["dst_v"], s["dst_acc"] = torch.zeros_like(s["dst_k"]), torch.zeros(dpages, Hkv, page, device=dev)
        return s
    drafts = _drafts(c)
    n, Hq = sum(drafts), c["Hq"]
    mask = _trees(drafts, rng)
    s["table"], pages = _pool(c, [a + t for a, t in zip(ctx, drafts)], g, dev)
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    s["cu"] = torch.tensor([0] + list(np.cumsum(drafts)), dtype=torch.int32, device=dev)
    s["k"], s["v"] = normal(pages, Hkv, page, D), normal(pages, Hkv, page, D)
    if c["op"] == "rope":
        # the projections' output: the heads of q, k and v side by side in each token's row
        s["qkv"] = normal(n, Hq + 2 * Hkv, D, dtype=DTYPES[c["src"]])
        depth = _depths(mask) if c["T"] <= 256 else np.concatenate([np.arange(t) for t in drafts])
        first = np.repeat(np.array(ctx), drafts)
        s["pos"] = torch.from_numpy((first + depth).astype(np.int32)).to(dev)
        i = np.arange(c["rot"] // 2, dtype=np.float64)
        s["inv_freq"] = torch.from_numpy(c["base"] ** (-2.0 * i / c["rot"]) / c["stretch"]).to(dev)
        s["mscale"] = 1.0 if c["stretch"] == 1.0 else 0.1 * math.log(c["stretch"]) + 1.0
        return s
    s["q"] = normal(n, Hq, D, scale=2.0)   # scores of standard deviation 2: some keys stand out
    s["mask"] = torch.from_numpy(mask).to(dev) if c["T"] > 1 else None
    if c["acc"]:
        s["acc"] = torch.empty(pages, Hkv, page, device=dev).uniform_(0.0, 0.1, generator=g)
        s["acc_out"] = torch.zeros_like(s["acc"])
    return s


DECAY = 0.98   # of the running attention weights


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        return _RUN_OWN[c["op"]](s, c)
    return _RUN_PLAIN[c["op"]](s, c)


def _slots(s, c, T):
    """(sequence, index among its drafts) of every token, and its page and row in the cache."""
    n = s["pos"].shape[0]
    tok = torch.arange(n, device=s["cu"].device)
    b = torch.searchsorted(s["cu"].long(), tok, right=True) - 1
    slot = s["ctx"].long()[b] + tok - s["cu"].long()[b]
    return s["table"].long()[b, slot // c["page"]], slot % c["page"]


def _rotate(x, cos, sin, rot, half):
    x = x.float()
    r, rest = x[..., :rot], x[..., rot:]
    if half:
        a, b = r[..., : rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, rest], -1)


def _plain_rope(s, c):
    Hq, Hkv = c["Hq"], c["Hkv"]
    q, k, v = s["qkv"].split([Hq, Hkv, Hkv], 1)
    angle = s["pos"].double()[:, None, None] * s["inv_freq"]      # far positions need 64 bits
    cos, sin = (angle.cos() * s["mscale"]).float(), (angle.sin() * s["mscale"]).float()
    page, row = _slots(s, c, c["T"])
    s["k"][page, :, row] = _rotate(k, cos, sin, c["rot"], c["half"]).to(s["k"].dtype)
    s["v"][page, :, row] = v.float().to(s["v"].dtype)
    return {"q": _rotate(q, cos, sin, c["rot"], c["half"]).to(s["k"].dtype), "k": s["k"], "v": s["v"]}


def _plain_tree(s, c):
    dev, (B, T, Hkv, D) = s["q"].device, (c["B"], c["T"], c["Hkv"], c["D"])
    G = c["Hq"] // Hkv
    cu, ctx, table = s["cu"].long(), s["ctx"].long(), s["table"].long()
    drafts = cu[1:] - cu[:-1]
    L = table.shape[1] * c["page"]
    # queries by sequence, padded to T; keys and values by sequence, padded to L
    j, l = torch.arange(T, device=dev), torch.arange(L, device=dev)
    live = j < drafts[:, None]
    at = torch.where(live, cu[:-1, None] + j, 0)
    qf = s["q"].float()[at].view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    kf = s["k"][table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D).float()
    x = torch.matmul(qf, kf.transpose(2, 3)).view(B, Hkv, T, G, L) * (1.0 / math.sqrt(D))
    del kf
    d = l - ctx[:, None]                                               # index among the drafts
    seen = (d < 0)[:, None].expand(B, T, L)
    inside = (d >= 0) & (d < drafts[:, None])
    if s["mask"] is None:
        seen = seen | (inside[:, None] & (d[:, None] <= j[:, None]))
    else:
        dd = d.clamp(0, 32 * s["mask"].shape[1] - 1)[:, None].expand(B, T, L)
        bit = (s["mask"][at].gather(2, dd >> 5) >> (dd & 31)) & 1
        seen = seen | (inside[:, None] & (bit == 1))
    seen = seen[:, None, :, None]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    del x
    z = p.sum(-1, keepdim=True)
    p = p / torch.where(z == 0, 1.0, z)
    vf = s["v"][table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D).float()
    vf = torch.where((l < (ctx + drafts)[:, None])[:, None, :, None], vf, 0.0)
    o = torch.matmul(p.view(B, Hkv, T * G, L), vf).view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4)
    lse = (top + z.log())[..., 0].permute(0, 2, 1, 3)
    out = {"o": o.reshape(B, T, c["Hq"], D)[live].to(DTYPES[c["out"]]), "lse": lse.reshape(B, T, c["Hq"])[live]}
    if c["acc"]:
        w = torch.where(live[:, None, :, None, None], p, 0.0).sum((2, 3))       # [B][Hkv][L]
        b, slot = torch.nonzero(l < (ctx + drafts)[:, None], as_tuple=True)
        page, row = table[b, slot // c["page"]], slot % c["page"]
        s["acc_out"][page, :, row] = DECAY * s["acc"][page, :, row] + w[b, :, slot]
        out["acc"] = s["acc_out"]
    return out


def _plain_evict(s, c):
    dev, (B, Hkv, page) = s["k"].device, (c["B"], c["Hkv"], c["page"])
    budget, table, lens = c["budget"], s["table"].long(), s["lens"].long()
    L = table.shape[1] * page
    l = torch.arange(L, device=dev)
    a = s["acc"][table].permute(0, 2, 1, 3).reshape(B, Hkv, L)
    fixed = (l < c["sink"]) | (l >= lens[:, None] - c["recent"])
    a = torch.where(fixed[:, None], math.inf, a)
    a = torch.where((l < lens[:, None])[:, None], a, -math.inf)
    if L < budget:
        a = torch.nn.functional.pad(a, (0, budget - L), value=-math.inf)
    ids = a.sort(dim=-1, descending=True, stable=True).indices[..., :budget]   # ties: the lowest first
    ids = torch.where(ids < lens[:, None, None], ids, a.shape[-1]).sort(-1).values
    new = lens.clamp(max=budget)
    b, h, i = torch.nonzero((torch.arange(budget, device=dev) < new[:, None])[:, None].expand(B, Hkv, budget),
                            as_tuple=True)
    src = ids[b, h, i]
    sp, sr = table[b, src // page], src % page
    dp, dr = s["dst_table"].long()[b, i // page], i % page
    for name in ("k", "v", "acc"):
        s["dst_" + name][dp, h, dr] = s[name][sp, h, sr]
    keep = torch.where(ids < lens[:, None, None], ids, -1).int()
    return {"keep": keep, "lens": new.int(), "k": s["dst_k"], "v": s["dst_v"], "acc": s["dst_acc"]}


def _own_rope(s, c):
    import int4_group_quantized_gs64_gb300 as qmv
    if "cache" not in s:
        s["cache"] = qmv.AttnCache(s["k"], s["v"])
    Hq, Hkv = c["Hq"], c["Hkv"]
    q, k, v = s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv], s["qkv"][:, Hq + Hkv:]
    out = qmv.attn_rope_append(s["cache"], q, k, v, s["pos"], s["inv_freq"], s["table"], s["ctx"], s["cu"],
                               interleaved=not c["half"], mscale=s["mscale"])
    return {"q": out, "k": s["k"], "v": s["v"]}


def _own_tree(s, c):
    import int4_group_quantized_gs64_gb300 as qmv
    if "cache" not in s:
        s["cache"] = qmv.AttnCache(s["k"], s["v"])
        n = qmv.attn_tree_workspace_bytes(s["cache"], c["Hq"], c["B"], s["q"].shape[0], c["T"],
                                          s["table"].shape[1], c["acc"])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=s["k"].device)
    o, lse = qmv.attn_tree(s["cache"], s["q"], s["table"], s["ctx"], s["cu"], c["T"], mask=s["mask"],
                           o_dtype=DTYPES[c["out"]], acc=s.get("acc"), acc_out=s.get("acc_out"), decay=DECAY,
                           ws=s["ws"])
    out = {"o": o, "lse": lse}
    if c["acc"]:
        out["acc"] = s["acc_out"]
    return out


def _own_evict(s, c):
    import int4_group_quantized_gs64_gb300 as qmv
    if "cache" not in s:
        s["cache"], s["dst"] = qmv.AttnCache(s["k"], s["v"]), qmv.AttnCache(s["dst_k"], s["dst_v"])
    keep, lens = qmv.attn_evict(s["cache"], s["acc"], s["table"], s["lens"], c["budget"], s["dst"], s["dst_acc"],
                                s["dst_table"], sink=c["sink"], recent=c["recent"])
    return {"keep": keep, "lens": lens, "k": s["dst_k"], "v": s["dst_v"], "acc": s["dst_acc"]}


_RUN_PLAIN = {"rope": _plain_rope, "tree": _plain_tree, "evict": _plain_evict}
_RUN_OWN = {"rope": _own_rope, "tree": _own_tree, "evict": _own_evict}


# ------------------------------------------------------------------ in 64 bits, one sequence at a time

def exact(c, seed):
    s = prepare(c, seed)
    return {"rope": _exact_rope, "tree": _exact_tree, "evict": _exact_evict}[c["op"]](s, c)


def _rows(pool, table_row, n):
    """The first n rows of a sequence in a pool: [n][Hkv][...] (a copy)."""
    p = pool[table_row.long()]
    return p.transpose(1, 2).reshape(-1, *p.shape[1:2], *p.shape[3:])[:n]


def _exact_rope(s, c):
    Hq, Hkv, rot = c["Hq"], c["Hkv"], c["rot"]
    k, v = s["k"].double(), s["v"].double()
    x = s["qkv"].double()
    turn = torch.polar(torch.full((1,), s["mscale"], dtype=torch.float64, device=x.device),
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


def _exact_tree(s, c):
    D, Hkv, page = c["D"], c["Hkv"], c["page"]
    G = c["Hq"] // Hkv
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=s["q"].device)
    acc = s["acc_out"].double() if c["acc"] else None
    words = s["mask"].cpu().numpy().view(np.uint8) if s["mask"] is not None else None
    for b in range(c["B"]):
        t, n = cu[b + 1] - cu[b], ctx[b] + cu[b + 1] - cu[b]
        see = np.ones((t, n), bool)
        if words is None:
            see[:, ctx[b]:] = np.tril(np.ones((t, t), bool))
        else:
            bits = np.unpackbits(words[cu[b]:cu[b + 1]], axis=1, bitorder="little")
            see[:, ctx[b]:] = bits[:, :t] == 1
        see = torch.from_numpy(see).to(o.device)
        row = s["table"][b]
        k, v = _rows(s["k"], row, n), _rows(s["v"], row, n)
        for h in range(Hkv):
            for g in range(G):
                x = s["q"][cu[b]:cu[b + 1], h * G + g].double() @ k[:, h].double().T / math.sqrt(D)
                x.masked_fill_(~see, -math.inf)
                e = torch.logsumexp(x, 1)
                x = torch.exp(x - e[:, None])
                o[cu[b]:cu[b + 1], h * G + g] = x @ v[:, h].double()
                lse[cu[b]:cu[b + 1], h * G + g] = e
                x = x.sum(0)
                if g == 0:
                    w = x
                else:
                    w = w + x
            if acc is not None:
                l = torch.arange(n, device=o.device)
                at = (row.long()[l // page], h, l % page)
                acc[at] = DECAY * s["acc"][at].double() + w
    return {"o": o, "lse": lse, "acc": acc} if c["acc"] else {"o": o, "lse": lse}


def _exact_evict(s, c):
    k, v, acc = s["dst_k"].double(), s["dst_v"].double(), s["dst_acc"].double()
    keep = torch.full((c["B"], c["Hkv"], c["budget"]), -1, dtype=torch.int32)
    lens = []
    for b, n in enumerate(s["lens"].tolist()):
        m = min(n, c["budget"])
        lens.append(m)
        a = _rows(s["acc"], s["table"][b], n).cpu().numpy()
        kk, vv, aa = (_rows(s[x], s["table"][b], n) for x in ("k", "v", "acc"))
        i = np.arange(m)
        for h in range(c["Hkv"]):
            ids = np.arange(n)
            if n > m:
                mid = ids[c["sink"]:n - c["recent"]]
                best = np.lexsort((mid, -a[mid, h].astype(np.float64)))[: m - c["sink"] - c["recent"]]
                ids = np.sort(np.concatenate([ids[:c["sink"]], mid[best], ids[n - c["recent"]:]]))
            keep[b, h, :m] = torch.from_numpy(ids.astype(np.int32))
            at = (s["dst_table"][b].long()[torch.from_numpy(i // c["page"]).to(k.device)], h,
                  torch.from_numpy(i % c["page"]).to(k.device))
            ids = torch.from_numpy(ids).to(k.device)
            k[at], v[at], acc[at] = kk[ids, h].double(), vv[ids, h].double(), aa[ids, h].double()
    return {"keep": keep, "lens": torch.tensor(lens, dtype=torch.int32), "k": k, "v": v, "acc": acc}
