"""Rotary append, tree attention and eviction on the GPU against plain 64-bit forms.

Tolerances are bounds, derived from the arithmetic: a rounding to a type is off
by at most eps / 2 relative to the value; a product of D terms in fp32
accumulators by D + 2 steps of 2^-23 of the sum of magnitudes (a tensor core may
cut instead of round); ex2 by 2^-22 relative."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
q = pytest.importorskip("int4_group_quantized_gs64_gb300")

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    q.build()
    q.lib()


def half_step(dt):
    return torch.finfo(dt).eps / 2


class Case:
    """A paged cache with shuffled pages, and a ragged batch of new tokens."""

    def __init__(self, ctx, drafts, Hkv=2, G=2, D=128, page=16, dtype=BF, seed=0, mask="tree",
                 qscale=1.0, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        self.ctx_l, self.drafts, self.Hkv, self.G, self.D, self.page = ctx, drafts, Hkv, G, D, page
        self.dtype, self.B, self.N, self.Hq = dtype, len(ctx), sum(drafts), Hkv * G
        need = [max(1, -(-(c + t) // page)) for c, t in zip(ctx, drafts)]
        self.width, pages = max(need), sum(need) + spare
        order = torch.randperm(pages, generator=g)[: sum(need)].tolist()
        table = torch.full((self.B, self.width), -7, dtype=torch.int32)  # unused entries: no page
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.table_l = table.tolist()

        def normal(*s, scale=1.0):
            return (torch.randn(*s, generator=g) * scale).to(dtype)

        self.k, self.v = normal(pages, Hkv, page, D), normal(pages, Hkv, page, D)
        self.q = normal(self.N, self.Hq, D, scale=qscale)
        self.acc = torch.rand(pages, Hkv, page, generator=g)
        self.T = max(drafts)
        self.table, self.cu_l = table, [0] + np.cumsum(drafts).tolist()
        if mask == "tree":
            W = -(-self.T // 32)
            rows = []
            for t in drafts:
                bits = []
                for j in range(t):
                    p = int(self.rng.integers(-1, j)) if j else -1
                    bits.append((bits[p] if p >= 0 else 0) | (1 << j))
                rows += [[(x >> (32 * w)) & 0xFFFFFFFF for w in range(W)] for x in bits]
            self.mask = torch.from_numpy(np.array(rows, np.uint32).reshape(self.N, W).view(np.int32))
        else:
            self.mask = None

    def dev(self):
        self.cache = q.AttnCache(self.k.cuda(), self.v.cuda())
        self.ctx = torch.tensor(self.ctx_l, dtype=torch.int32).cuda()
        self.cu = torch.tensor(self.cu_l, dtype=torch.int32).cuda()
        return self

    def seen(self, b):
        """[T][len] truth table of what each draft sees."""
        t, n = self.drafts[b], self.ctx_l[b] + self.drafts[b]
        s = np.ones((t, n), bool)
        if self.mask is None:
            s[:, self.ctx_l[b]:] = np.tril(np.ones((t, t), bool))
        else:
            w = self.mask.numpy().view(np.uint32)[self.cu_l[b]:self.cu_l[b + 1]]
            for i in range(t):
                for d in range(t):
                    s[i, self.ctx_l[b] + d] = (int(w[i, d // 32]) >> (d % 32)) & 1
        return torch.from_numpy(s)

    def rows(self, pool, b, h):
        n = self.ctx_l[b] + self.drafts[b]
        j = np.arange(n)
        pg = torch.tensor([self.table_l[b][x // self.page] for x in j], dtype=torch.long)
        return pool[pg, h, torch.from_numpy(j % self.page)].double()

    def reference(self, scale, decay=1.0, acc_in=None):
        """o, lse, weights in 64 bits, and the bounds of o (before its rounding), lse and weights."""
        D, dev = self.D, "cuda"
        o = torch.zeros(self.N, self.Hq, D, dtype=torch.float64)
        ob, lse = torch.zeros_like(o), torch.full((self.N, self.Hq), -math.inf, dtype=torch.float64)
        lb = torch.zeros_like(lse)
        acc = torch.zeros(self.k.shape[:3], dtype=torch.float64) if acc_in is None else acc_in.double().clone()
        touched = torch.zeros(acc.shape, dtype=torch.bool)
        ab = torch.zeros_like(acc)
        for b in range(self.B):
            if self.drafts[b] == 0:
                continue
            see, n = self.seen(b).to(dev), self.ctx_l[b] + self.drafts[b]
            sl = slice(self.cu_l[b], self.cu_l[b + 1])
            j = np.arange(n)
            pg = torch.tensor([self.table_l[b][x // self.page] for x in j], dtype=torch.long)
            rw = torch.from_numpy(j % self.page)
            for h in range(self.Hkv):
                k, v = self.rows(self.k, b, h).to(dev), self.rows(self.v, b, h).to(dev)
                w = torch.zeros(n, dtype=torch.float64, device=dev)
                wb = torch.zeros_like(w)
                for g in range(self.G):
                    hq = h * self.G + g
                    qq = self.q[sl, hq].double().to(dev)
                    kk = torch.where(see.any(0)[:, None], k, 0.0)   # unseen keys may hold anything
                    x = (qq @ kk.T) * scale
                    mag = ((qq.abs() @ kk.abs().T) * abs(scale)).masked_fill(~see, 0.0)
                    x = x.masked_fill(~see, -math.inf)
                    e = torch.logsumexp(x, 1)
                    none = e == -math.inf
                    p = torch.exp(x - torch.where(none, 0.0, e)[:, None])
                    p = torch.where(see & ~none[:, None], p, 0.0)
                    vv = torch.where(see.any(0)[:, None], v, 0.0)
                    # a score's error: D + 2 steps of its magnitude, and the scaling's roundings
                    ds = mag.amax(1) * (D + 6) * 2.0 ** -23 + 2.0 ** -22
                    rel = 2 * ds + (n + 8) * 2.0 ** -24 + 2.0 ** -21
                    o[sl, hq] = (p @ vv).cpu()
                    ob[sl, hq] = ((p @ vv.abs()) * rel[:, None]).cpu()
                    lse[sl, hq], lb[sl, hq] = e.cpu(), (ds + rel + torch.where(none, 0.0, e).abs() * 2.0 ** -22).cpu()
                    w += p.sum(0)
                    wb += (p * rel[:, None]).sum(0)
                wb += w * self.N * 2.0 ** -23
                acc[pg, h, rw] = decay * acc[pg, h, rw] + w.cpu()
                ab[pg, h, rw] = wb.cpu() + acc[pg, h, rw].abs() * 2.0 ** -22
                touched[pg, h, rw] = True
        return o, ob, lse, lb, acc, ab, touched


def check_tree(c, o, lse, ref, p_round):
    """p_round: how much of each weight its rounding may be off on the way to the product."""
    eo, ob, el, lb = ref[:4]
    mag = ob + 0
    dt = o.dtype
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.equal(torch.isinf(lse), torch.isinf(el))
    fin = torch.isfinite(el)
    assert torch.all((lse - el)[fin].abs() <= lb[fin]), float(((lse - el)[fin].abs() - lb[fin]).max())
    tol = mag + p_round + eo.abs() * half_step(dt) + 2.0 ** -24
    bad = (o - eo).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((o - eo).abs() / tol).max()))


def p_rounding(c, scale, dt):
    """Bound from the weights' own rounding: a 16-bit output may round each weight once
    (half a step), an fp32 output carries them as two 16-bit numbers (half a step squared)."""
    hs = half_step(c.dtype)
    f = hs * hs * 2 if dt == F32 else hs
    out = torch.zeros(c.N, c.Hq, c.D, dtype=torch.float64)
    for b in range(c.B):
        if c.drafts[b] == 0:
            continue
        see = c.seen(b)
        sl = slice(c.cu_l[b], c.cu_l[b + 1])
        for h in range(c.Hkv):
            k, v = c.rows(c.k, b, h), c.rows(c.v, b, h)
            k, v = (torch.where(see.any(0)[:, None], x, 0.0).cuda() for x in (k, v))
            for g in range(c.G):
                x = (c.q[sl, h * c.G + g].double().cuda() @ k.T) * scale
                p = torch.softmax(x.masked_fill(~see.cuda(), -1e300), 1)
                out[sl, h * c.G + g] = ((p @ v.abs()) * f * 2).cpu()   # numerator and sum
    return out


def run_tree(c, o_dtype=None, scale=None, **kw):
    c.dev()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = q.attn_tree(c.cache, c.q.cuda(), c.table.cuda(), c.ctx, c.cu, max(c.T, 1),
                         mask=None if c.mask is None else c.mask.cuda(), o_dtype=o_dtype,
                         scale=scale, status=st, **kw)
    torch.cuda.synchronize()
    assert int(st) == 0
    return o, lse


SHAPES = [
    # ctx, drafts, Hkv, G, D, page, dtype, mask
    ([5], [1], 1, 1, 64, 16, BF, None),
    ([0], [1], 1, 1, 128, 16, BF, None),
    ([0, 15, 16, 17, 63, 64, 65], [1] * 7, 2, 4, 128, 16, BF, None),
    ([1, 127, 128, 129, 1000], [1] * 5, 1, 8, 64, 32, FP, None),
    ([777], [1], 8, 6, 128, 64, BF, None),
    ([300, 0, 41], [4, 0, 3], 2, 4, 128, 64, FP, "tree"),
    ([33, 250], [3, 5], 2, 3, 64, 128, BF, "tree"),
    ([64, 100, 7], [8, 7, 1], 1, 4, 128, 256, FP, "tree"),
    ([500, 13], [31, 33], 2, 2, 128, 16, BF, "tree"),
    ([90, 0], [64, 40], 1, 8, 128, 32, BF, "tree"),
    ([200], [100], 2, 5, 64, 16, FP, "tree"),
    ([130], [65], 1, 7, 128, 64, BF, None),
    ([10], [256], 1, 2, 64, 64, BF, "tree"),
    ([5000, 4000], [1, 1], 2, 16, 128, 64, BF, None),
    ([3000], [2], 4, 16, 64, 64, FP, "tree"),
    ([2000, 10, 900], [17, 20, 2], 2, 8, 128, 128, FP, "tree"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
@pytest.mark.parametrize("out", ["same", "fp32"])
def test_tree_shapes(shape, out):
    ctx, drafts, Hkv, G, D, page, dt, mask = shape
    c = Case(ctx, drafts, Hkv, G, D, page, dt, seed=len(ctx) + D, mask=mask, qscale=2.0)
    odt = F32 if out == "fp32" else dt
    o, lse = run_tree(c, o_dtype=odt)
    s = D ** -0.5
    check_tree(c, o, lse, c.reference(s), p_rounding(c, s, odt))


def test_tree_long_context_split_over_blocks():
    for Hkv, G, T in ((1, 4, 1), (2, 6, 9)):
        c = Case([70001], [T], Hkv, G, 128, 64, BF, seed=T, qscale=2.0)
        o, lse = run_tree(c, o_dtype=F32)
        s = 128 ** -0.5
        check_tree(c, o, lse, c.reference(s), p_rounding(c, s, F32))


@pytest.mark.parametrize("D,page,G,T", [(128, 128, 5, 21), (128, 64, 5, 21), (128, 16, 8, 16),
                                        (64, 128, 5, 21), (128, 128, 8, 40), (64, 32, 8, 40)])
def test_tree_batches_bound_by_memory(D, page, G, T):
    """Long contexts of many sequences: copies arrive late and rings run dry. Every
    sequence's values are compared, on the GPU, in 64 bits."""
    B, Hkv, n = 12, 8, 6000
    g = torch.Generator(device="cuda").manual_seed(T)
    ctx = [n - 211 * b for b in range(B)]
    drafts = [T - b % 3 for b in range(B)]
    need = [-(-(c + t) // page) for c, t in zip(ctx, drafts)]
    k = torch.empty(sum(need), Hkv, page, D, dtype=BF, device="cuda").normal_(generator=g)
    v = torch.empty_like(k).normal_(generator=g)
    table = torch.zeros(B, max(need), dtype=torch.int32)
    order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(1)).int()
    for b in range(B):
        table[b, :need[b]] = order[sum(need[:b]):sum(need[:b + 1])]
    cu = [0] + np.cumsum(drafts).tolist()
    qq = torch.empty(cu[-1], Hkv * G, D, dtype=BF, device="cuda").normal_(generator=g)
    cache = q.AttnCache(k, v)
    i32 = dict(dtype=torch.int32, device="cuda")
    acc = torch.zeros(k.shape[:3], device="cuda")
    st = torch.zeros(1, **i32)
    runs = [q.attn_tree(cache, qq, table.cuda(), torch.tensor(ctx, **i32), torch.tensor(cu, **i32), T,
                        acc_out=acc, status=st) for _ in range(4)]
    torch.cuda.synchronize()
    assert int(st) == 0
    for o, lse in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])
    o, lse = runs[0]
    for b in range(B):
        t, m = drafts[b], ctx[b] + drafts[b]
        rows = table[b, :need[b]].long().cuda()
        kk = k[rows].transpose(1, 2).reshape(-1, Hkv, D)[:m].double()
        vv = v[rows].transpose(1, 2).reshape(-1, Hkv, D)[:m].double()
        x = torch.einsum("thgd,mhd->htgm", qq[cu[b]:cu[b + 1]].view(t, Hkv, G, D).double(), kk) * D ** -0.5
        late = torch.arange(m, device="cuda") > ctx[b] + torch.arange(t, device="cuda")[:, None]
        x.masked_fill_(late[None, :, None], -math.inf)
        e = x.logsumexp(-1)
        p = torch.exp(x - e[..., None])
        want = torch.einsum("htgm,mhd->thgd", p, vv).reshape(t, Hkv * G, D)
        mag = torch.einsum("htgm,mhd->thgd", p, vv.abs()).reshape(t, Hkv * G, D)
        # half a step of the weights (numerator and sum) and of the output, scores' errors beside them
        tol = mag * (2 * half_step(BF) + 2.0 ** -14) + want.abs() * half_step(BF)
        assert torch.all((o[cu[b]:cu[b + 1]].double() - want).abs() <= tol), b
        assert torch.allclose(lse[cu[b]:cu[b + 1]].double(), e.permute(1, 0, 2).reshape(t, -1), atol=2.0 ** -14, rtol=0)
        w = acc[rows].transpose(1, 2).reshape(-1, Hkv)[:m].double()
        assert torch.allclose(w, p.sum((1, 2)).T, rtol=2.0 ** -13, atol=1e-9), b


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D,page,G,T", [(128, 64, 5, 1), (64, 64, 4, 4), (128, 16, 5, 21), (64, 128, 5, 21),
                                        (128, 128, 8, 40), (64, 32, 8, 40)])
def test_tree_fp32_outputs_of_long_contexts(D, page, G, T, dtype):
    """An fp32 output is as near as fp32 weights and sums are. In the norm: a score
    (rms 1) off by up to 10 steps of 2^-24, a weight by about that much, each by
    itself (1.2e-6); a tile's 24 partial products cut by 2^-25 on average, all one
    way (7e-7). Together under 2^-19."""
    B, Hkv, n = 9, 4, 5000
    g = torch.Generator(device="cuda").manual_seed(T + D)
    ctx, drafts = [n - 411 * b for b in range(B)], [max(1, T - b % 3) for b in range(B)]
    need = [-(-(c + t) // page) for c, t in zip(ctx, drafts)]
    k = torch.empty(sum(need), Hkv, page, D, dtype=dtype, device="cuda").normal_(generator=g)
    v = torch.empty_like(k).normal_(generator=g)
    table = torch.zeros(B, max(need), dtype=torch.int32)
    order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(1)).int()
    for b in range(B):
        table[b, :need[b]] = order[sum(need[:b]):sum(need[:b + 1])]
    cu = [0] + np.cumsum(drafts).tolist()
    qq = torch.empty(cu[-1], Hkv * G, D, dtype=dtype, device="cuda").normal_(generator=g)
    i32 = dict(dtype=torch.int32, device="cuda")
    st = torch.zeros(1, **i32)
    runs = [q.attn_tree(q.AttnCache(k, v), qq, table.cuda(), torch.tensor(ctx, **i32), torch.tensor(cu, **i32), T,
                        o_dtype=F32, status=st) for _ in range(3)]
    torch.cuda.synchronize()
    assert int(st) == 0
    for o, lse in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])
    for b in range(B):
        t, m = drafts[b], ctx[b] + drafts[b]
        rows = table[b, :need[b]].long().cuda()
        kk = k[rows].transpose(1, 2).reshape(-1, Hkv, D)[:m].double()
        vv = v[rows].transpose(1, 2).reshape(-1, Hkv, D)[:m].double()
        x = torch.einsum("thgd,mhd->htgm", qq[cu[b]:cu[b + 1]].view(t, Hkv, G, D).double(), kk) * D ** -0.5
        late = torch.arange(m, device="cuda") > ctx[b] + torch.arange(t, device="cuda")[:, None]
        want = torch.einsum("htgm,mhd->thgd", torch.softmax(x.masked_fill(late[None, :, None], -math.inf), -1), vv)
        got = runs[0][0][cu[b]:cu[b + 1]].double().view_as(want)
        assert (got - want).norm() <= 2.0 ** -19 * want.norm(), b


def test_tree_peaked_scores_and_negative_scale():
    """Scores of tens of units, rising and falling along the keys: the running maximum moves."""
    for scale in (1.0, -0.5):
        c = Case([900], [3], 2, 4, 64, 16, FP, seed=3, qscale=1.5)
        o, lse = run_tree(c, o_dtype=F32, scale=scale)
        check_tree(c, o, lse, c.reference(scale), p_rounding(c, scale, F32))


@pytest.mark.parametrize("T,G", [(4, 2), (40, 8)])
def test_tree_rows_that_see_nothing(T, G):
    c = Case([0, 50], [T, T], 2, G, 128, 16, BF, seed=1)
    c.mask[1] = 0            # nothing cached, nothing allowed: an empty row
    c.mask[T + 2] = 0        # the cache alone
    o, lse = run_tree(c)
    s = 128 ** -0.5
    check_tree(c, o, lse, c.reference(s), p_rounding(c, s, BF))
    assert torch.all(o[1] == 0) and torch.all(lse[1] == -math.inf)


@pytest.mark.parametrize("T,G,dt", [(5, 2, BF), (5, 2, FP), (48, 4, BF), (48, 4, FP)])
def test_tree_infinities_and_nans_in_places_not_seen(T, G, dt):
    """Stale slots after the end, unused pages and masked drafts hold anything."""
    c = Case([37, 0], [T, T], 1, G, 64, 32, dt, seed=2)
    clean = Case([37, 0], [T, T], 1, G, 64, 32, dt, seed=2)
    held = torch.zeros(c.k.shape[0], 32, dtype=torch.bool)
    for b in range(2):
        for j in range(c.ctx_l[b] + T):
            held[c.table_l[b][j // 32], j % 32] = True
    rng = np.random.default_rng(0)
    for pool in (c.k, c.v):
        junk = torch.from_numpy(rng.choice([math.nan, math.inf, -math.inf], size=pool.shape)).to(dt)
        pool.copy_(torch.where(held[:, None, :, None], pool, junk))
    # draft 3 of both sequences is seen by itself alone, and is not finite
    bad = 3
    for cc in (c, clean):
        for b in range(2):
            for t in range(T):
                if t != bad:
                    cc.mask[b * T + t, bad // 32] &= ~(1 << (bad % 32))
    for b in range(2):
        j = c.ctx_l[b] + bad
        pg, rw = c.table_l[b][j // 32], j % 32
        c.v[pg, 0, rw, 0::3] = math.inf
        c.v[pg, 0, rw, 1::3] = math.nan
        c.k[pg, 0, rw, 5] = math.nan if b else 0.0
    o, lse = run_tree(c)
    oc, lc = run_tree(clean)
    others = [n for n in range(2 * T) if n % T != bad]
    assert torch.equal(o[others], oc[others]) and torch.equal(lse[others], lc[others])
    # the row that sees it: infinities and NaNs where the value has them (all NaN where its key is)
    assert torch.all(torch.isnan(o[T + bad])) and torch.all(torch.isnan(lse[T + bad]))
    assert torch.all(~torch.isfinite(o[bad][:, 0::3])) and torch.all(torch.isnan(o[bad][:, 1::3]))
    assert torch.all(torch.isfinite(o[bad][:, 2::3]))


@pytest.mark.parametrize("drafts,G,D", [([1, 1], 4, 128), ([5, 3], 3, 64), ([20, 7], 8, 128), ([70, 64], 5, 64)])
def test_tree_weights(drafts, G, D):
    c = Case([333, 20], drafts, 2, G, D, 32, BF, seed=5, qscale=2.0)
    s = D ** -0.5
    o0, l0 = run_tree(c)
    # out of place with a decay
    acc, out = c.acc.cuda(), torch.full(c.acc.shape, 5.0, device="cuda")
    o, lse = run_tree(c, acc=acc, acc_out=out, decay=0.75)
    assert torch.equal(o, o0) and torch.equal(lse, l0) and torch.equal(acc.cpu(), c.acc)
    ref = c.reference(s, 0.75, c.acc)
    t = ref[6]
    assert torch.all((out.cpu().double() - ref[4])[t].abs() <= ref[5][t])
    assert torch.all(out.cpu()[~t] == 5.0)       # slots of no sequence are not touched
    # in place, and from nothing
    run_tree(c, acc=acc, decay=0.75)
    assert torch.equal(acc.cpu()[t], out.cpu()[t]) and torch.equal(acc.cpu()[~t], c.acc[~t])
    out2 = torch.full(c.acc.shape, 5.0, device="cuda")
    run_tree(c, acc_out=out2)
    ref = c.reference(s, 1.0, torch.zeros_like(c.acc))
    assert torch.all((out2.cpu().double() - ref[4])[t].abs() <= ref[5][t])


@pytest.mark.parametrize("drafts,G,D", [([200, 3], 8, 128), ([256, 130], 5, 64), ([65, 64], 8, 128)])
def test_tree_weights_of_many_rows(drafts, G, D):
    """More rows than a pass over the keys holds, and sequences that have none in the later passes."""
    c = Case([300, 45], drafts, 2, G, D, 32, BF, seed=6, qscale=2.0)
    acc, out = c.acc.cuda(), torch.full(c.acc.shape, 5.0, device="cuda")
    run_tree(c, acc=acc, acc_out=out, decay=0.75)
    assert torch.equal(acc.cpu(), c.acc)
    ref = c.reference(D ** -0.5, 0.75, c.acc)
    t = ref[6]
    assert torch.all((out.cpu().double() - ref[4])[t].abs() <= ref[5][t])
    assert torch.all(out.cpu()[~t] == 5.0)
    run_tree(c, acc=acc, decay=0.75)  # in place
    assert torch.equal(acc.cpu()[t], out.cpu()[t]) and torch.equal(acc.cpu()[~t], c.acc[~t])


@pytest.mark.parametrize("drafts,G,D,width", [([4, 3], 4, 128, 16400), ([1, 1], 1, 64, 262200), ([2, 2], 3, 64, 43700)])
def test_tree_weights_of_few_rows_in_wide_tables(drafts, G, D, width):
    """Tables so wide that the scores of a call are not kept."""
    c = Case([700, 20], drafts, 2, G, D, 256, BF, seed=7, qscale=2.0)
    more = torch.full((2, width - c.table.shape[1]), -7, dtype=torch.int32)
    c.table = torch.cat([c.table, more], 1).contiguous()
    c.dev()
    assert q.attn_tree_workspace_bytes(c.cache, c.Hq, 2, c.N, c.T, width, True) < 1 << 29
    out = torch.full(c.acc.shape, 5.0, device="cuda")
    run_tree(c, acc=c.acc.cuda(), acc_out=out, decay=0.75)
    ref = c.reference(D ** -0.5, 0.75, c.acc)
    t = ref[6]
    assert torch.all((out.cpu().double() - ref[4])[t].abs() <= ref[5][t])
    assert torch.all(out.cpu()[~t] == 5.0)


def test_tree_weights_of_rows_that_see_nothing():
    c = Case([0], [4], 1, 2, 64, 16, BF, seed=1)
    c.mask[:] = 0
    out = torch.full(c.acc.shape, 5.0, device="cuda")
    run_tree(c, acc_out=out)
    pg = c.table_l[0][0]
    assert torch.all(out[pg, :, :4] == 0) and torch.all(out[pg, :, 4:] == 5.0)


def test_tree_strided_queries_streams_graph_and_same_bits():
    c = Case([3000, 40, 700], [9, 9, 2], 2, 4, 128, 64, BF, seed=8, qscale=2.0).dev()
    wide = torch.randn(c.N, c.Hq + 4, 128).to(BF).cuda()
    wide[:, 2:2 + c.Hq] = c.q.cuda()
    view = wide[:, 2:2 + c.Hq]
    args = (c.table.cuda(), c.ctx, c.cu, c.T)
    kw = dict(mask=c.mask.cuda())
    o0, l0 = q.attn_tree(c.cache, c.q.cuda(), *args, **kw)
    o1, l1 = q.attn_tree(c.cache, view, *args, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, l2 = q.attn_tree(c.cache, view, *args, stream=s, **kw)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(o0, o1) and torch.equal(l0, l1) and torch.equal(o0, o2) and torch.equal(l0, l2)
    ws = torch.empty(q.attn_tree_workspace_bytes(c.cache, c.Hq, c.B, c.N, c.T, c.width), dtype=torch.uint8, device="cuda")
    o3, l3 = torch.zeros_like(o0), torch.zeros_like(l0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.attn_tree(c.cache, view, *args, o=o3, lse=l3, ws=ws, **kw)
    for _ in range(3):
        ws.fill_(255)
        o3.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o3, o0) and torch.equal(l3, l0)


@pytest.mark.parametrize("T,G", [(3, 2), (40, 4)])
def test_tree_bad_pages_and_lengths_are_left_out(T, G):
    c = Case([100, 90, 60], [T, T, T], 2, G, 64, 16, FP, seed=4)
    s = 64 ** -0.5
    # page 2 of sequence 0 names no page: its 16 tokens are not seen
    table = c.table.clone()
    table[0, 2] = c.k.shape[0] + 5
    c.dev()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(c.acc.shape, device="cuda")
    o, lse = q.attn_tree(c.cache, c.q.cuda(), table.cuda(), c.ctx, c.cu, T, mask=c.mask.cuda(), status=st,
                         acc_out=out)
    torch.cuda.synchronize()
    assert int(st) == 1
    seen = c.seen

    def without(b):
        m = seen(b)
        if b == 0:
            m[:, 32:48] = False
        return m
    c.seen = without
    ref = c.reference(s)
    check_tree(c, o, lse, ref, p_rounding(c, s, FP))
    c.seen = seen
    # a length that does not fit its row of the table, and more drafts than the bound
    for ctx, md, left in (([100, 10 ** 6, 60], T, 1), ([100, -1, 60], T, 1)):
        st.zero_()
        o2 = torch.full_like(o, 9.0)
        q.attn_tree(c.cache, c.q.cuda(), c.table.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(), c.cu, md,
                    mask=c.mask.cuda(), status=st, o=o2)
        torch.cuda.synchronize()
        assert int(st) == 2
        assert torch.all(o2[left * T:(left + 1) * T] == 9.0)
        full, _ = q.attn_tree(c.cache, c.q.cuda(), c.table.cuda(), c.ctx, c.cu, T, mask=c.mask.cuda())
        keep = [n for n in range(3 * T) if n // T != left]
        p = p_rounding(c, s, FP)
        ref = c.reference(s)
        assert torch.all((o2[keep].double().cpu() - ref[0][keep]).abs() <=
                         ref[1][keep] + p[keep] + ref[0][keep].abs() * half_step(FP) + 2.0 ** -24)


# ------------------------------------------------------------------ rotary positions and append

ROPE = [
    # ctx, drafts, Hkv, G, D, page, cache, input, rot, interleaved
    ([0], [1], 1, 1, 64, 16, BF, BF, 64, False),
    ([5000], [1], 8, 6, 128, 64, BF, BF, 128, False),
    ([7, 0, 250], [3, 0, 70], 2, 3, 128, 16, FP, F32, 64, True),
    ([100000, 31], [5, 2], 2, 2, 64, 32, BF, F32, 32, False),
    ([15, 16], [17, 300], 1, 4, 128, 128, FP, FP, 128, True),
    ([3], [9], 2, 2, 64, 16, FP, F32, 50, False),       # rot no multiple of 16
    ([3], [9], 2, 2, 64, 16, BF, BF, 6, True),
    ([3], [9], 2, 2, 128, 16, BF, BF, 2, False),
]


def rope_reference(x, pos, inv_freq, rot, inter, m):
    x = x.double()
    ang = torch.outer(pos.double(), inv_freq)[:, None]
    cos, sin = ang.cos() * m, ang.sin() * m
    y = x.clone()
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., i], x[..., j]
    y[..., i], y[..., j] = a * cos - b * sin, b * cos + a * sin
    bound = torch.zeros_like(x)
    # cos and sin: the fraction's rounding (2^-24 of a turn), two steps of sincospi, mscale's and the products'
    e = (a.abs() + b.abs()) * m * (2 * math.pi * 2.0 ** -24 + 2.0 ** -21)
    bound[..., i] = e
    bound[..., j] = e
    return y, bound


@pytest.mark.parametrize("shape", ROPE, ids=[str(i) for i in range(len(ROPE))])
def test_rope_append(shape):
    ctx, drafts, Hkv, G, D, page, dt, src, rot, inter = shape
    c = Case(ctx, drafts, Hkv, G, D, page, dt, seed=rot).dev()
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(c.N, c.Hq + 2 * Hkv, D, generator=g).to(src)
    pos = torch.randint(0, 1 << 20, (c.N,), generator=g, dtype=torch.int32)
    inv = torch.tensor([10000.0 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    m = 1.25 if inter else 1.0
    d = qkv.cuda()
    acc = c.acc.cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = q.attn_rope_append(c.cache, d[:, :c.Hq], d[:, c.Hq:c.Hq + Hkv], d[:, c.Hq + Hkv:], pos.cuda(), inv.cuda(),
                             c.table.cuda(), c.ctx, c.cu, interleaved=inter, mscale=m, acc=acc, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    y, bound = rope_reference(qkv[:, :c.Hq + Hkv], pos, inv, rot, inter, m)
    tol = bound + y.abs() * half_step(dt) + 2.0 ** -25
    assert torch.all((out.double().cpu() - y[:, :c.Hq]).abs() <= tol[:, :c.Hq])
    k, v, a = c.cache.k.cpu(), c.cache.v.cpu(), acc.cpu()
    new = torch.zeros(k.shape[0], page, dtype=torch.bool)
    for b in range(c.B):
        for t in range(drafts[b]):
            s, n = ctx[b] + t, c.cu_l[b] + t
            pg, rw = c.table_l[b][s // page], s % page
            assert torch.all((k[pg, :, rw].double() - y[n, c.Hq:]).abs() <= tol[n, c.Hq:])
            assert torch.equal(v[pg, :, rw], qkv[n, c.Hq + Hkv:].to(dt))
            assert torch.all(a[pg, :, rw] == 0)
            new[pg, rw] = True
    old = ~new[:, None, :].expand(-1, Hkv, -1)
    assert torch.equal(k[old], c.k[old]) and torch.equal(v[old], c.v[old]) and torch.equal(a[old], c.acc[old])


@pytest.mark.parametrize("shift", [0, 2, 5])
def test_rope_strides_and_alignment(shift):
    """q, k and v as parts of wider rows, at any element offset."""
    c = Case([20], [11], 2, 2, 64, 16, BF, seed=shift).dev()
    g = torch.Generator().manual_seed(2)
    row = (c.Hq + 4) * 64 + 13
    flat = torch.randn(c.N * row + 64, generator=g).to(BF).cuda()
    view = flat[shift:shift + c.N * row].as_strided((c.N, c.Hq + 4, 64), (row, 64, 1), shift)
    pos = torch.arange(c.N, dtype=torch.int32).cuda() * 1000
    inv = torch.tensor([1000.0 ** (-i / 32) for i in range(32)], dtype=torch.float64).cuda()
    args = (pos, inv, c.table.cuda(), c.ctx, c.cu)
    o0 = q.attn_rope_append(c.cache, view[:, :4], view[:, 4:6], view[:, 6:], *args)
    k0, v0 = c.cache.k.clone(), c.cache.v.clone()
    t = view.contiguous()
    o1 = q.attn_rope_append(c.cache, t[:, :4], t[:, 4:6], t[:, 6:], *args)
    torch.cuda.synchronize()
    assert torch.equal(o0, o1) and torch.equal(k0, c.cache.k) and torch.equal(v0, c.cache.v)


def test_rope_bad_pages_and_lengths():
    c = Case([20, 8], [4, 4], 1, 2, 64, 16, BF, seed=0).dev()
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(c.N, c.Hq + 2, 64, generator=g).to(BF).cuda()
    pos, inv = torch.zeros(c.N, dtype=torch.int32).cuda(), torch.ones(32, dtype=torch.float64).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(table, ctx):
        st.zero_()
        k0 = c.cache.k.clone()
        o = q.attn_rope_append(c.cache, qkv[:, :2], qkv[:, 2:3], qkv[:, 3:], pos, inv, table, ctx, c.cu, status=st)
        torch.cuda.synchronize()
        return int(st), (c.cache.k != k0).flatten(1).any(1).nonzero().flatten().tolist(), o
    t = c.table.clone()
    t[0, 1] = -1
    s, changed, _ = call(t.cuda(), c.ctx)
    assert s == 1 and changed == [c.table_l[1][0]]
    c.cache.k.copy_(c.k)
    s, changed, _ = call(c.table.cuda(), torch.tensor([20, 10 ** 9], dtype=torch.int32).cuda())
    assert s == 2 and changed == [c.table_l[0][1]]


# ------------------------------------------------------------------ eviction

def evict_reference(c, lens, acc, budget, sink, recent):
    keep = -np.ones((c.B, c.Hkv, budget), np.int32)
    for b, n in enumerate(lens):
        for h in range(c.Hkv):
            a = np.array([acc[c.table_l[b][j // c.page], h, j % c.page] for j in range(n)], np.float64)
            if n <= budget:
                keep[b, h, :n] = np.arange(n)
                continue
            a = np.where(np.isnan(a), -np.inf, a)
            lowest = np.isnan([acc[c.table_l[b][j // c.page], h, j % c.page] for j in range(n)])
            mid = np.arange(sink, n - recent)
            order = mid[np.lexsort((mid, lowest[mid], -a[mid]))][: budget - sink - recent]
            keep[b, h] = np.sort(np.concatenate([np.arange(sink), order, np.arange(n - recent, n)]))
    return keep


EVICT = [
    # lens, budget, sink, recent, Hkv, D, page, dst page, dtype
    ([100], 30, 2, 5, 2, 64, 16, 16, BF),
    ([1, 0, 40, 41], 40, 0, 0, 1, 128, 16, 32, FP),
    ([500, 64, 333], 64, 4, 60, 2, 64, 32, 64, BF),      # sink + recent fill the budget
    ([4099, 37], 1024, 4, 128, 2, 128, 64, 128, BF),
    ([20011], 777, 16, 100, 3, 64, 128, 16, FP),
    ([70003], 5000, 1, 0, 1, 64, 64, 64, BF),            # a cluster of blocks a list
    ([9], 1, 0, 0, 1, 64, 16, 16, BF),
    ([9], 1, 1, 0, 1, 64, 16, 16, BF),
    ([9], 1, 0, 1, 1, 64, 16, 16, BF),
]


@pytest.mark.parametrize("shape", EVICT, ids=[str(i) for i in range(len(EVICT))])
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_evict(shape, kind):
    lens, budget, sink, recent, Hkv, D, page, dpage, dt = shape
    c = Case(lens, [0] * len(lens), Hkv, 1, D, page, dt, seed=budget, mask=None).dev()
    rng = np.random.default_rng(budget)
    if kind == "spread":
        acc = np.exp(rng.normal(size=c.acc.shape) * 3).astype(np.float32)
    elif kind == "ties":
        acc = rng.integers(0, 3, size=c.acc.shape).astype(np.float32)
    else:
        acc = rng.choice(np.array([0.0, -0.0, np.nan, np.inf, -np.inf, 1e-40, -1.0, 3.0], np.float32), size=c.acc.shape)
    dp = -(-budget // dpage)
    order = torch.randperm(c.B * dp + 2)[: c.B * dp].view(c.B, dp).int()
    dst = q.AttnCache(torch.full((c.B * dp + 2, Hkv, dpage, D), 3.0, dtype=dt).cuda(),
                      torch.full((c.B * dp + 2, Hkv, dpage, D), 4.0, dtype=dt).cuda())
    dacc = torch.full((c.B * dp + 2, Hkv, dpage), 5.0).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = torch.from_numpy(acc)
    keep, new = q.attn_evict(c.cache, a.cuda(), c.table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), budget,
                             dst, dacc, order.cuda(), sink=sink, recent=recent, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    want = evict_reference(c, lens, acc, budget, sink, recent)
    assert np.array_equal(keep.cpu().numpy(), want)
    assert new.tolist() == [min(n, budget) for n in lens]
    ek = torch.full_like(dst.k, 3.0).cpu(); ev = torch.full_like(dst.v, 4.0).cpu()
    ea = torch.full_like(dacc, 5.0).cpu()
    for b, n in enumerate(lens):
        m = min(n, budget)
        i = torch.arange(m)
        to = order[b].long()[i // dpage]
        for h in range(Hkv):
            s = torch.from_numpy(want[b, h, :m]).long()
            pg = torch.tensor(c.table_l[b])[s // page].long()
            ek[to, h, i % dpage] = c.k[pg, h, s % page]
            ev[to, h, i % dpage] = c.v[pg, h, s % page]
            ea[to, h, i % dpage] = a[pg, h, s % page]
    assert torch.equal(dst.k.cpu(), ek) and torch.equal(dst.v.cpu(), ev)
    assert np.array_equal(dacc.cpu().numpy(), ea.numpy(), equal_nan=True)


def test_evict_bad_pages_and_lengths():
    c = Case([50, 50], [0, 0], 1, 1, 64, 16, BF, seed=0, mask=None).dev()
    dst, dacc = q.AttnCache.empty(4, 1, 16, 64), torch.zeros(4, 1, 16).cuda()
    dst.k.zero_()
    dt = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = c.table.clone()
    t[0, 0] = 10 ** 6
    lens = torch.tensor([50, 10 ** 7], dtype=torch.int32).cuda()
    keep, new = q.attn_evict(c.cache, torch.ones_like(c.acc).cuda(), t.cuda(), lens, 20, dst, dacc, dt, sink=3, status=st)
    torch.cuda.synchronize()
    assert int(st) == 3 and new.tolist() == [20, 0] and torch.all(keep[1] == -1)
    # its own tokens have the lowest sums, so the first 17 with a page are kept beside the sink
    assert keep[0, 0].tolist() == [0, 1, 2] + list(range(16, 33))
    assert torch.all(dst.k[0, 0, :3] == 0)      # nowhere to read them from: not written


# ------------------------------------------------------------------ together

def test_steps_of_a_cache_that_is_evicted():
    """Prompt in, decode steps with running weights, eviction, and a step over what is left."""
    torch.manual_seed(0)
    B, Hkv, G, D, page = 2, 2, 4, 64, 16
    cache = q.AttnCache.empty(64, Hkv, page, D, torch.bfloat16)
    cache.k.zero_(); cache.v.zero_()
    acc = torch.full((64, Hkv, page), 77.0, device="cuda")
    table = torch.arange(32, dtype=torch.int32, device="cuda").view(B, 16)
    inv = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).cuda()
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 100, 180], dtype=torch.int32, device="cuda")
    lens = [100, 80]
    for step in range(4):
        if step:
            cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
        n = int(cu[-1])
        pos = torch.cat([torch.arange(int(cu[b + 1] - cu[b])) + int(ctx[b]) for b in range(B)]).int().cuda()
        x = torch.randn(n, Hkv * (G + 2), D, device="cuda")
        qq = q.attn_rope_append(cache, x[:, :Hkv * G], x[:, Hkv * G:Hkv * (G + 1)], x[:, Hkv * (G + 1):], pos, inv,
                                table, ctx, cu, acc=acc)
        o, lse = q.attn_tree(cache, qq, table, ctx, cu, 100 if step == 0 else 1, acc=acc, decay=0.9)
        ctx += cu[1:] - cu[:-1]
    torch.cuda.synchronize()
    assert torch.isfinite(o.float()).all()
    # every row's weights sum to one: 3 decode steps and the prompt, decayed
    total = [sum(0.9 ** (3 - s) * G * (lens[b] if s == 0 else 1) for s in range(4)) for b in range(B)]
    for b in range(B):
        got = acc[table[b].long()].permute(1, 0, 2).reshape(Hkv, -1)[:, : int(ctx[b])].double().sum(1)
        assert torch.allclose(got, torch.full_like(got, total[b]), rtol=1e-4)
    dst_table = torch.arange(32, 36, dtype=torch.int32, device="cuda").view(B, 2)
    keep, new = q.attn_evict(cache, acc, table, ctx, 32, cache, acc, dst_table, sink=2, recent=8)
    o2, _ = q.attn_tree(cache, qq, dst_table, new - 1, cu, 1)
    for b in range(B):
        for h in range(Hkv):
            s = keep[b, h].long()
            pg = table[b].long()[s // page]
            k, v = cache.k[pg, h, s % page].double(), cache.v[pg, h, s % page].double()
            p = torch.softmax(qq[b, h * G:(h + 1) * G].double() @ k.T * D ** -0.5, 1)
            assert torch.allclose(o2[b, h * G:(h + 1) * G].double(), p @ v, atol=2.0 ** -7, rtol=0)


# ------------------------------------------------------------------ many sequences, short items

def check_batch(ctx, drafts, Hkv, G, D, page, dtype, out=None, weights=True, runs=3):
    """A batch of any number of sequences against 64 bits on the GPU, a chain each; repeats are bit-equal."""
    g = torch.Generator(device="cuda").manual_seed(len(ctx) + D)
    B, T = len(ctx), max(drafts)
    need = [-(-(c + t) // page) for c, t in zip(ctx, drafts)]
    k = torch.empty(sum(need), Hkv, page, D, dtype=dtype, device="cuda").normal_(generator=g)
    v = torch.empty_like(k).normal_(generator=g)
    table = torch.full((B, max(need)), -3, dtype=torch.int32)
    order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(1)).int()
    at = np.concatenate([[0], np.cumsum(need)])
    for b in range(B):
        table[b, :need[b]] = order[at[b]:at[b + 1]]
    cu = [0] + np.cumsum(drafts).tolist()
    qq = torch.empty(cu[-1], Hkv * G, D, dtype=dtype, device="cuda").normal_(generator=g)
    i32 = dict(dtype=torch.int32, device="cuda")
    st, cache = torch.zeros(1, **i32), q.AttnCache(k, v)
    args = (qq, table.cuda(), torch.tensor(ctx, **i32), torch.tensor(cu, **i32), T)
    first = None
    for _ in range(runs):
        acc = torch.full(k.shape[:3], 7.0, device="cuda")
        o, lse = q.attn_tree(cache, *args, o_dtype=out, acc_out=acc if weights else None, status=st)
        torch.cuda.synchronize()
        assert int(st) == 0
        if first is None:
            first = (o, lse, acc)
        assert all(torch.equal(x, y) for x, y in zip(first, (o, lse, acc)))
    o, lse, acc = first
    hs = half_step(o.dtype)
    for b in range(B):
        t, m = drafts[b], ctx[b] + drafts[b]
        rows = table[b, :need[b]].long().cuda()
        kk = k[rows].transpose(1, 2).reshape(-1, Hkv, D)[:m].double()
        vv = v[rows].transpose(1, 2).reshape(-1, Hkv, D)[:m].double()
        w = acc[rows].transpose(1, 2).reshape(-1, Hkv).double()
        if t == 0:
            assert torch.all(w == 7)       # no step: its sums stay as they are
            continue
        x = torch.einsum("thgd,mhd->htgm", qq[cu[b]:cu[b + 1]].view(t, Hkv, G, D).double(), kk) * D ** -0.5
        late = torch.arange(m, device="cuda") > ctx[b] + torch.arange(t, device="cuda")[:, None]
        x.masked_fill_(late[None, :, None], -math.inf)
        e = x.logsumexp(-1)
        p = torch.exp(x - e[..., None])
        want = torch.einsum("htgm,mhd->thgd", p, vv).reshape(t, Hkv * G, D)
        mag = torch.einsum("htgm,mhd->thgd", p, vv.abs()).reshape(t, Hkv * G, D)
        # the weights' roundings (numerator and sum), scores of rms 1 off by up to 2^-15, the output's rounding
        tol = mag * (2 * half_step(dtype) + 2.0 ** -14) + want.abs() * hs
        assert torch.all((o[cu[b]:cu[b + 1]].double() - want).abs() <= tol), b
        assert torch.allclose(lse[cu[b]:cu[b + 1]].double(), e.permute(1, 0, 2).reshape(t, -1), atol=2.0 ** -14, rtol=0), b
        if weights:
            assert torch.allclose(w[:m], p.sum((1, 2)).T, rtol=2.0 ** -13, atol=1e-9), b
            assert torch.all(w[m:] == 7), b


@pytest.mark.parametrize("D,dtype,out", [(128, BF, BF), (64, FP, FP), (128, FP, F32), (128, BF, F32)])
def test_tree_many_short_items(D, dtype, out):
    """Items of one key tile and of two, several of them a block: a stream has none in some."""
    ctx = [[90, 30, 200, 0, 101, 250][b % 6] for b in range(120)]
    check_batch(ctx, [5 + b % 3 for b in range(120)], 4, 4, D, 32, dtype, out, weights=False)


@pytest.mark.parametrize("D,page,dtype", [(128, 64, BF), (64, 32, FP)])
def test_tree_weights_of_four_row_tiles_over_long_contexts(D, page, dtype):
    """385 to 512 rows: four products a key tile, score buffers used over and over, ring of two slots."""
    check_batch([2500 - 171 * b for b in range(12)], [64 - b % 16 for b in range(12)], 8, 8, D, page, dtype)


def test_tree_weights_of_ragged_row_tiles():
    """One to four products a tile, parts of one tile and of many in a block."""
    check_batch([[120, 40, 700, 3][b % 4] for b in range(60)], [[64, 5, 33, 20, 50][b % 5] for b in range(60)],
                4, 8, 128, 64, BF)


@pytest.mark.parametrize("D,G,big", [(128, 8, 100), (64, 5, 250)])
def test_tree_weights_of_ragged_batches_beyond_one_launch(D, G, big):
    """A few large trees among many small ones: most sequences have no rows beyond the first 512."""
    check_batch([[70, 900, 130, 20][b % 4] for b in range(64)], [big if b % 21 == 3 else 3 for b in range(64)],
                8, G, D, 32, BF)


# ------------------------------------------------------------------ first tokens out of order

@pytest.mark.parametrize("cu,ctx", [([0, 10, 20, 0, 30], [0, 30, 0, 0]), ([5, 10, 0, 10], [0, 0, 0]),
                                    ([3, 7, 7, 2], [4, 9, 0]), ([-4, 6, 12], [3, 8]), ([0, 9, 40, 12], [0, 2, 5])])
@pytest.mark.parametrize("rot", [32, 6])
def test_rope_first_tokens_out_of_order(cu, ctx, rot):
    """A token goes to the last sequence that holds it and nowhere else; sequences of negative length
    or beyond N are left out. (A guard page on each side of the sequences' own stays as it was.)"""
    B, Hkv, G, D, page, N = len(ctx), 2, 2, 64, 16, 30 if max(cu) > 20 else 12
    c = Case([48] * B, [0] * B, Hkv, G, D, page, BF, seed=B, mask=None, spare=6).dev()
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(N, c.Hq + 2 * Hkv, D, generator=g).to(BF).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    # the table in the middle of a larger one: what lies beside it names pages too
    pages = c.k.shape[0]
    used = {p for r in c.table_l for p in r}
    free = [p for p in range(pages) if p not in used]
    wide = torch.tensor([[free[0]] * 3] * 2 + c.table_l + [[free[1]] * 3] * 2, **i32)
    table = wide[2:2 + B]
    st = torch.zeros(1, **i32)
    q.attn_rope_append(c.cache, qkv[:, :c.Hq], qkv[:, c.Hq:c.Hq + Hkv], qkv[:, c.Hq + Hkv:],
                       torch.zeros(N, **i32), torch.ones(rot // 2, dtype=torch.float64, device="cuda"), table,
                       torch.tensor(ctx, **i32), torch.tensor(cu, **i32), status=st)
    torch.cuda.synchronize()
    assert int(st) == 2
    want = c.v.clone()
    for n in range(N):
        held = [b for b in range(B) if cu[b] <= n < cu[b + 1]]
        if held and cu[held[-1]] >= 0 and cu[held[-1] + 1] <= N:
            b = held[-1]
            slot = ctx[b] + n - cu[b]
            want[c.table_l[b][slot // page], :, slot % page] = qkv[n, c.Hq + Hkv:].cpu()
    assert torch.equal(c.cache.v.cpu(), want)


def test_rope_many_sequences():
    """More than 32 sequences, some without tokens."""
    lens = [(7 * b) % 50 for b in range(150)]
    drafts = [b % 4 for b in range(150)]
    c = Case(lens, drafts, 2, 2, 64, 16, FP, seed=1, mask=None).dev()
    g = torch.Generator().manual_seed(6)
    qkv = torch.randn(c.N, c.Hq + 4, 64, generator=g).to(FP).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = q.attn_rope_append(c.cache, qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], torch.zeros(c.N, dtype=torch.int32).cuda(),
                             torch.ones(32, dtype=torch.float64).cuda(), c.table.cuda(), c.ctx, c.cu, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0 and torch.equal(out, qkv[:, :4])      # positions 0: nothing turns
    k, v = c.k.clone(), c.v.clone()
    for b in range(c.B):
        for t in range(drafts[b]):
            s = lens[b] + t
            k[c.table_l[b][s // 16], :, s % 16] = qkv[c.cu_l[b] + t, 4:6].cpu()
            v[c.table_l[b][s // 16], :, s % 16] = qkv[c.cu_l[b] + t, 6:].cpu()
    assert torch.equal(c.cache.k.cpu(), k) and torch.equal(c.cache.v.cpu(), v)


# ------------------------------------------------------------------ infinities in cached keys and values

@pytest.mark.parametrize("T,G,D", [(1, 4, 64), (7, 3, 64), (5, 8, 128), (20, 8, 128)])
def test_tree_weights_with_infinite_keys(T, G, D):
    """A cached key that scores -inf in every row adds no weight, whatever the number of rows (queries
    beside the last row's must not add a NaN); the others' weights are those without it."""
    c = Case([150, 40], [T, T], 2, G, D, 16, BF, seed=11, qscale=2.0, mask=None)
    c.q[..., 0] = c.q[..., 0].abs() + 0.5
    spot = [(0, 17), (1, 0), (0, 149)]
    for b, j in spot:
        c.k[c.table_l[b][j // 16], :, j % 16] = 0.0
        c.k[c.table_l[b][j // 16], :, j % 16, 0] = -math.inf
    out = torch.full(c.acc.shape, 5.0, device="cuda")
    o, lse = run_tree(c, acc=c.acc.cuda(), acc_out=out, decay=0.5)
    for b, j in spot:   # 64-bit form: such keys are not seen
        c.k[c.table_l[b][j // 16], :, j % 16] = 0.0
    seen = c.seen

    def without(b):
        m = seen(b)
        for bb, j in spot:
            if bb == b:
                m[:, j] = False
        return m
    c.seen = without
    s = D ** -0.5
    ref = c.reference(s, 0.5, c.acc)
    check_tree(c, o, lse, ref, p_rounding(c, s, BF))
    t = ref[6]
    assert torch.all((out.cpu().double() - ref[4])[t].abs() <= ref[5][t])


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("T,G,D,ctx", [(1, 4, 64, 40), (2, 4, 128, 3000), (20, 8, 128, 40), (9, 4, 64, 3000),
                                       (40, 8, 128, 300), (40, 8, 64, 300)])
def test_tree_rows_of_scores_minus_inf(T, G, D, ctx, out):
    """A row whose keys all score -inf gets zeros, whatever the values are, one block a row or several."""
    c = Case([ctx], [T], 1, G, D, 64, BF, seed=12)
    c.q[..., 0] = c.q[..., 0].abs() + 0.5
    c.k.zero_()
    c.k[..., 0] = -math.inf
    c.v[:, :, ::3] = math.inf
    c.v[:, :, 1::3, ::2] = math.nan
    weights = torch.full(c.acc.shape, 5.0, device="cuda")
    o, lse = run_tree(c, o_dtype=out, acc=c.acc.cuda(), acc_out=weights)
    assert torch.all(o == 0) and torch.all(lse == -math.inf)
    held = torch.zeros(c.k.shape[0], 64, dtype=torch.bool)
    for j in range(ctx + T):
        held[c.table_l[0][j // 64], j % 64] = True
    held = held[:, None].expand(-1, 1, -1)
    assert torch.equal(weights.cpu()[held], c.acc[held])


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("out", ["same", "fp32"])
@pytest.mark.parametrize("T,G,D,ctx", [(1, 4, 64, 0), (3, 4, 128, 37), (3, 4, 128, 200), (20, 8, 128, 37), (40, 8, 64, 130)])
def test_tree_infinite_values_of_drafts_that_are_seen(T, G, D, ctx, out, dt):
    """An infinity among a seen draft's values is the output's too, where nothing else moves it: also in a
    row's first keys, and where the draft's score is far above the keys' before it."""
    c = Case([ctx], [T], 1, G, D, 16, dt, seed=13, mask=None)
    c.q[..., 0] = 30.0
    c.k[..., 0] = -30.0 if ctx else 1.0
    j = ctx
    pg, rw = c.table_l[0][j // 16], j % 16
    c.k[pg, 0, rw, 0] = 30.0       # the first draft, which every row sees, has by far the largest score
    c.v[pg, 0, rw, 0::2] = math.inf
    c.v[pg, 0, rw, 1] = -math.inf
    o, lse = run_tree(c, o_dtype=F32 if out == "fp32" else dt, scale=1.0)
    assert torch.isfinite(lse).all()
    assert torch.all(o[..., 0::2] == math.inf) and torch.all(o[..., 1] == -math.inf)
    assert torch.isfinite(o[..., 3::2]).all()


@pytest.mark.parametrize("T,G", [(1, 4), (6, 8)])
def test_tree_pages_that_sequences_share(T, G):
    """Without running weights sequences may share the pages of a common prefix."""
    c = Case([200, 170, 300], [T] * 3, 2, G, 64, 32, BF, seed=21, qscale=2.0)
    o0, l0 = run_tree(c)
    table, k, v = c.table.clone(), c.k.clone(), c.v.clone()
    for b in (1, 2):        # the first 160 tokens are sequence 0's
        for i in range(5):
            k[c.table_l[b][i]], v[c.table_l[b][i]] = c.k[c.table_l[0][i]], c.v[c.table_l[0][i]]
            table[b, i] = c.table_l[0][i]
    own, shared = c.table, table
    c.k, c.v = k, v
    apart = run_tree(c)
    c.table = shared
    together = run_tree(c)
    c.table = own
    assert torch.equal(apart[0], together[0]) and torch.equal(apart[1], together[1])
    assert torch.equal(apart[0][:T], o0[:T]) and torch.equal(apart[1][:T], l0[:T])


@pytest.mark.parametrize("T,G", [(1, 4), (6, 8), (70, 8)])
def test_tree_weights_of_sequences_without_new_tokens(T, G):
    """A sequence that takes no step keeps its sums, without a decay."""
    c = Case([200, 170, 90], [T, 0, T], 2, G, 64, 32, BF, seed=22, mask=None)
    out = torch.full(c.acc.shape, 5.0, device="cuda")
    run_tree(c, acc=c.acc.cuda(), acc_out=out, decay=0.5)
    ref = c.reference(64 ** -0.5, 0.5, c.acc)
    t = ref[6]
    assert torch.all((out.cpu().double() - ref[4])[t].abs() <= ref[5][t])
    assert torch.all(out.cpu()[~t] == 5.0)
    for p in c.table_l[1][:6]:
        assert torch.all(out[p] == 5.0)


def test_calls_leave_the_current_device():
    c = Case([30], [1], 1, 2, 64, 16, BF, seed=25, mask=None)
    before = torch.cuda.current_device()
    run_tree(c)
    with pytest.raises(TypeError):
        q.attn_tree(c.cache, c.q, c.table.cuda(), c.ctx, c.cu, 1)    # refused in the middle of its checks
    assert torch.cuda.current_device() == before


@pytest.mark.parametrize("rot,inter", [(64, False), (32, True), (6, False)])
def test_rope_positions_to_the_ends_of_int32(rot, inter):
    """Negative positions and those near 2^31: the angle's bound grows with the position."""
    edge = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, -2 ** 30 - 7, 2 ** 30 + 1, 123456789, -1, -99999, 0, 1]
    c = Case([0], [len(edge)], 1, 2, 64, 16, FP, seed=26, mask=None).dev()
    g = torch.Generator().manual_seed(7)
    qkv = torch.randn(c.N, 4, 64, generator=g)
    pos = torch.tensor(edge, dtype=torch.int32)
    inv = torch.tensor([10000.0 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    d = qkv.cuda()
    out = q.attn_rope_append(c.cache, d[:, :2], d[:, 2:3], d[:, 3:], pos.cuda(), inv.cuda(), c.table.cuda(), c.ctx,
                             c.cu, interleaved=inter)
    y, bound = rope_reference(qkv[:, :3], pos, inv, rot, inter, 1.0)
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    x = qkv[:, :3].double()
    # 3 roundings of 2^-53 here, and one in the reference's own product
    more = (x[..., i].abs() + x[..., j].abs()) * torch.outer(pos.double().abs(), inv)[:, None] * 4 * 2.0 ** -53
    bound[..., i] += more
    bound[..., j] += more
    tol = bound + y.abs() * half_step(FP) + 2.0 ** -25
    assert torch.all((out.double().cpu() - y[:, :2]).abs() <= tol[:, :2])
    k = torch.stack([c.cache.k[c.table_l[0][s // 16], 0, s % 16] for s in range(c.N)]).double().cpu()
    assert torch.all((k - y[:, 2]).abs() <= tol[:, 2])


@pytest.mark.parametrize("T,G", [(3, 2), (40, 4)])
def test_tree_more_drafts_than_the_bound(T, G):
    """A sequence with more drafts than max_draft is left out; the others are as ever."""
    c = Case([100, 90, 60], [T - 1, T, T - 1], 2, G, 64, 16, FP, seed=23)
    full, lse = run_tree(c)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, l = torch.full_like(full, 9.0), torch.full_like(lse, 9.0)
    acc = torch.full(c.acc.shape, 5.0, device="cuda")
    q.attn_tree(c.cache, c.q.cuda(), c.table.cuda(), c.ctx, c.cu, T - 1, mask=c.mask.cuda(), status=st, o=o, lse=l,
                acc_out=acc)
    torch.cuda.synchronize()
    assert int(st) == 2
    left = slice(T - 1, 2 * T - 1)
    assert torch.all(o[left] == 9.0) and torch.all(l[left] == 9.0)
    for p in c.table_l[1][: (90 + T + 15) // 16]:
        assert torch.all(acc[p] == 5.0)
    keep = [n for n in range(c.N) if not T - 1 <= n < 2 * T - 1]
    e, le = full[keep].double(), lse[keep].double()
    # the same keys in other shares: a few steps of fp32 apart, and each a rounding of the output
    assert torch.all((o[keep].double() - e).abs() <= e.abs() * 2 * half_step(FP) + 2.0 ** -12)
    assert torch.all((l[keep].double() - le).abs() <= 2.0 ** -18 * (1 + le.abs()))


# ------------------------------------------------------------------ eviction of many long lists

@pytest.mark.parametrize("kind", ["spread", "ties", "equal"])
def test_evict_more_lists_than_sms_longer_than_a_block_keeps(kind):
    """160 lists of up to 45,000 sums: a block a list, whose last slots are read again from memory."""
    B, Hkv, D, page, n = 20, 8, 64, 64, 45000
    lens = [n - 137 * b for b in range(B)]
    budget, sink, recent = 4100, 5, 333
    g = torch.Generator(device="cuda").manual_seed(3)
    need = [-(-x // page) for x in lens]
    table = torch.zeros(B, max(need), dtype=torch.int32)
    order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(1)).int()
    at = np.concatenate([[0], np.cumsum(need)])
    for b in range(B):
        table[b, :need[b]] = order[at[b]:at[b + 1]]
    src = q.AttnCache.empty(sum(need), Hkv, page, D)
    src.k.view(torch.int16).random_(generator=g)
    src.v.view(torch.int16).random_(generator=g)
    acc = torch.empty(sum(need), Hkv, page, device="cuda")
    if kind == "spread":
        acc.normal_(0.0, 2.0, generator=g).exp_()
    elif kind == "ties":
        acc.random_(0, 7, generator=g)
    else:
        acc.fill_(0.25)
    dp = -(-budget // page)
    dst, dacc = q.AttnCache.empty(B * dp, Hkv, page, D), torch.full((B * dp, Hkv, page), 9.0, device="cuda")
    dt = torch.arange(B * dp, dtype=torch.int32, device="cuda").view(B, dp)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep, new = q.attn_evict(src, acc, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), budget,
                             dst, dacc, dt, sink=sink, recent=recent, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0 and new.tolist() == [budget] * B
    i = torch.arange(budget, device="cuda")
    for b in range(B):
        rows, m = table[b, :need[b]].long().cuda(), lens[b]
        a = acc[rows].transpose(0, 1).reshape(Hkv, -1)[:, :m]
        mid = a[:, sink:m - recent].sort(dim=-1, descending=True, stable=True).indices[:, :budget - sink - recent] + sink
        fixed = torch.cat([torch.arange(sink, device="cuda"), torch.arange(m - recent, m, device="cuda")])
        want = torch.cat([mid, fixed.expand(Hkv, -1)], 1).sort(-1).values
        assert torch.equal(keep[b].long(), want), b
        h = torch.arange(Hkv, device="cuda")[:, None]
        pg, to = rows[want // page], dt[b].long()[i // page].expand(Hkv, -1)
        for x, y in ((src.k, dst.k), (src.v, dst.v)):
            assert torch.equal(x[pg, h, want % page].view(torch.int16), y[to, h, i % page].view(torch.int16)), b
        assert torch.equal(acc[pg, h, want % page], dacc[to, h, i % page]), b


# ------------------------------------------------------------------ batches of more than 32 sequences

@pytest.mark.parametrize("D,dtype,drafts,G", [(128, BF, [1], 4), (64, FP, [1, 0, 2], 5), (128, FP, [1, 3, 0, 2], 4),
                                              (64, BF, [30, 7, 0, 1], 5), (128, BF, [40, 1], 8)])
@pytest.mark.parametrize("B", [33, 300])
def test_tree_batches_of_many_sequences(D, dtype, drafts, G, B):
    """Shares counted by the whole block, several sequences a thread, some without tokens."""
    check_batch([(b * 71) % 640 for b in range(B)], [drafts[b % len(drafts)] for b in range(B)], 2, G, D, 32, dtype,
                runs=2)
