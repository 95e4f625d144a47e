"""Windowed attention on the GPU against a plain 64-bit form, with the bounds of the tree
attention's tests (test_gpu_attn): they hold for any set of keys that a row sees."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
q = pytest.importorskip("int4_group_quantized_gs64_gb300")

from test_gpu_attn import BF, FP, F32, Case, check_tree, half_step, p_rounding  # noqa: E402

pytestmark = pytest.mark.gpu
ALL = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    q.build()
    q.lib()


class Win(Case):
    """Chains whose tokens see a window and some first slots; pages that none of a sequence's
    new tokens sees are not in its table, and what no token sees holds NaNs."""

    def __init__(self, ctx, new, W, S, Hkv=2, G=2, D=128, page=16, dtype=BF, seed=0, qscale=2.0):
        super().__init__(ctx, new, Hkv, G, D, page, dtype, seed, mask=None, qscale=qscale)
        self.W, self.S = W, S
        poison = torch.ones(self.k.shape[0], page, dtype=torch.bool)
        for b in range(self.B):
            some = self.seen(b).any(0)
            for j in range(len(some)):
                if some[j]:
                    poison[self.table_l[b][j // page], j % page] = False
            for i in range(self.width):
                if not some[i * page:(i + 1) * page].any():
                    self.table_l[b][i] = -3 - i
        self.table = torch.tensor(self.table_l, dtype=torch.int32)
        bad = poison[:, None, :, None].expand_as(self.k)
        self.k[bad], self.v[bad] = math.nan, math.nan

    def rows(self, pool, b, h):
        n = self.ctx_l[b] + self.drafts[b]
        j = np.arange(n)
        pg = torch.tensor([max(0, self.table_l[b][x // self.page]) for x in j], dtype=torch.long)
        x = pool[pg, h, torch.from_numpy(j % self.page)].double()
        return torch.where(self.seen(b).any(0)[:, None], x, 0.0)

    def seen(self, b):
        p = np.arange(self.ctx_l[b], self.ctx_l[b] + self.drafts[b])[:, None]
        j = np.arange(self.ctx_l[b] + self.drafts[b])[None]
        return torch.from_numpy((j <= p) & ((p - j < self.W) | (j < self.S)))


def run(c, o_dtype=None, scale=None, max_new=None, **kw):
    c.dev()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = q.attn_window(c.cache, c.q.cuda(), c.table.cuda(), c.ctx, c.cu, max_new or c.T,
                           window=None if c.W == ALL else c.W, sinks=c.S, o_dtype=o_dtype, scale=scale, status=st, **kw)
    torch.cuda.synchronize()
    assert int(st) == 0
    return o, lse


SHAPES = [
    # ctx, new, window, sinks, Hkv, G, D, page, dtype
    ([0], [1], 1, 0, 1, 1, 64, 16, BF),
    ([5], [1], 3, 1, 1, 1, 128, 16, BF),
    ([0, 15, 16, 17, 63, 64, 65, 300], [1] * 8, 17, 4, 2, 4, 128, 16, BF),
    ([1000, 129, 0], [1, 1, 1], 100, 130, 1, 8, 64, 32, FP),
    ([4000], [1], 512, 4, 8, 6, 128, 64, BF),
    ([4000], [1], ALL, 0, 2, 16, 128, 64, BF),
    ([500, 0, 41], [4, 0, 3], 7, 2, 2, 4, 128, 64, FP),
    ([33, 250], [3, 5], 40, 17, 2, 3, 64, 128, BF),
    ([333], [7], 1, 0, 3, 2, 64, 16, BF),
    ([900, 13], [5, 1], 64, 64, 2, 3, 64, 256, FP),
    # more than 16 rows
    ([0], [300], ALL, 0, 2, 2, 128, 16, BF),
    ([0], [300], 64, 4, 2, 2, 128, 16, BF),
    ([1000, 10, 129], [33, 40, 1], 100, 3, 2, 8, 128, 32, BF),
    ([700], [100], 1, 0, 2, 5, 64, 16, FP),
    ([130, 2000], [65, 20], 256, 130, 1, 7, 128, 64, BF),
    ([0, 77, 0], [513, 1, 129], 128, 0, 1, 3, 64, 128, BF),
    ([2000, 10, 900], [17, 20, 2], 700, 16, 2, 2, 128, 128, FP),
    ([1500], [257], 513, 200, 1, 1, 128, 256, BF),
    ([60], [40], 2000, 4, 1, 300, 64, 16, BF),
    ([0], [1100], 300, 5, 1, 6, 128, 64, FP),
    ([3000, 0], [64, 64], 130, 1, 4, 1, 64, 64, FP),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
@pytest.mark.parametrize("out", ["same", "fp32"])
def test_shapes(shape, out):
    ctx, new, W, S, Hkv, G, D, page, dt = shape
    c = Win(ctx, new, W, S, Hkv, G, D, page, dt, seed=len(ctx) + D)
    odt = F32 if out == "fp32" else dt
    o, lse = run(c, o_dtype=odt)
    s = D ** -0.5
    check_tree(c, o, lse, c.reference(s), p_rounding(c, s, odt))


@pytest.mark.parametrize("T,G,max_new", [(1, 4, 1), (1, 4, 40), (2, 6, 300)])
def test_the_bound_chooses_the_kernel_not_the_result(T, G, max_new):
    """The same calls through the kernels for few and for many rows."""
    c = Win([1000, 30, 5000], [T, 1, T], 600, 4, 2, G, 128, 64, BF, seed=T)
    o, lse = run(c, o_dtype=F32, max_new=max_new)
    s = 128 ** -0.5
    check_tree(c, o, lse, c.reference(s), p_rounding(c, s, F32))


@pytest.mark.parametrize("Hkv,G,T,W,S", [(1, 4, 1, ALL, 0), (2, 6, 9, ALL, 0), (1, 2, 3, 30000, 70),
                                         (1, 3, 90, 40000, 4)])
def test_long_contexts_split_over_blocks(Hkv, G, T, W, S):
    c = Win([70001], [T], W, S, Hkv, G, 128, 64, BF, seed=T)
    o, lse = run(c, o_dtype=F32)
    s = 128 ** -0.5
    check_tree(c, o, lse, c.reference(s), p_rounding(c, s, F32))


@pytest.mark.parametrize("B,new", [(40, 1), (300, 2), (70, 20), (40, 130)])
def test_batches_of_many_sequences(B, new):
    """More sequences than a warp counts at once, some without new tokens."""
    rng = np.random.default_rng(B)
    ctx = rng.integers(0, 700, B).tolist()
    t = [0 if b % 7 == 3 else int(rng.integers(1, new + 1)) for b in range(B)]
    c = Win(ctx, t, 130, 4, 1, 4, 64, 16, BF, seed=B)
    o, lse = run(c)
    check_tree(c, o, lse, c.reference(0.125), p_rounding(c, 0.125, BF))


@pytest.mark.parametrize("T,G", [(3, 2), (40, 4)])
def test_scales(T, G):
    for scale in (-0.3, 0.0, 1.5):
        c = Win([60, 0], [T, T], 33, 2, 2, G, 64, 16, BF, seed=T, qscale=1.0)
        o, lse = run(c, scale=scale)
        check_tree(c, o, lse, c.reference(scale), p_rounding(c, scale, BF))


@pytest.mark.parametrize("T,G,dt", [(3, 4, BF), (3, 4, FP), (150, 2, BF), (40, 4, FP)])
@pytest.mark.parametrize("out", ["same", "fp32"])
def test_infinities_of_values_reach_those_that_see_them(T, G, dt, out):
    """A slot with infinite and NaN values: tokens whose window has passed it, and those before
    it, are as if it held zeros there; the others' elements are infinite or NaN."""
    W, S, D = 20, 3, 64
    c = Win([50, 7], [T, T], W, S, 1, G, D, 16, dt, seed=T)
    clean = c.v.clone()
    marks = [(0, 2, math.inf), (0, 50 - W + 2, math.nan), (0, 51, -math.inf), (1, 8, math.inf)]
    hit = torch.zeros(c.N, D, dtype=torch.bool)
    for i, (b, j, x) in enumerate(marks):
        pg, rw = c.table_l[b][j // 16], j % 16
        c.v[pg, :, rw, 5 * i + 1] = x
        clean[pg, :, rw, 5 * i + 1] = 0
        hit[c.cu_l[b]:c.cu_l[b + 1], 5 * i + 1] |= c.seen(b)[:, j]
    odt = F32 if out == "fp32" else dt
    o, lse = run(c, o_dtype=odt)
    o = o.cpu()
    hit = hit[:, None].expand(-1, c.Hq, -1)
    assert not torch.isfinite(o[hit]).any() and torch.isfinite(o[~hit]).all()
    c.v = clean
    ref, s = c.reference(D ** -0.5), D ** -0.5
    # (the zeros' weights are part of the sum either way)
    o[hit] = ref[0][hit].to(odt)
    check_tree(c, o, lse, ref, p_rounding(c, s, odt))


@pytest.mark.parametrize("T,G", [(3, 2), (40, 8)])
def test_rows_of_scores_minus_inf_and_hidden_keys(T, G):
    """A sequence whose visible keys all score -inf: zeros. Keys that hold infinities and NaNs and
    are hidden change nothing (they do in every case here: hidden slots hold NaNs)."""
    c = Win([40, 25], [T, T], 1, 0, 2, G, 64, 16, BF, seed=T, qscale=1.0)
    c.q[c.cu_l[1]:] = c.q[c.cu_l[1]:].abs() + 0.5
    for j in range(25, 25 + T):
        c.k[c.table_l[1][j // 16], :, j % 16] = -math.inf
    o, lse = run(c)
    o, lse = o.cpu(), lse.cpu()
    assert not o[c.cu_l[1]:].any() and torch.all(lse[c.cu_l[1]:] == -math.inf)
    ref = c.reference(0.125)
    n = c.cu_l[1]
    tol = ref[1][:n] + p_rounding(c, 0.125, BF)[:n] + ref[0][:n].abs() * half_step(BF) + 2.0 ** -24
    assert torch.all((o[:n].double() - ref[0][:n]).abs() <= tol)


@pytest.mark.parametrize("T,G,D", [(2, 4, 128), (60, 4, 128), (60, 2, 64)])
def test_strides_streams_graph_and_same_bits(T, G, D):
    c = Win([900, 33], [T, T - 1], 300, 4, 2, G, D, 32, BF, seed=T)
    c.k, c.v = c.k.nan_to_num(0.5), c.v.nan_to_num(0.5)   # (shorter contexts below see other slots)
    c.dev()
    args = [c.table.cuda(), c.ctx, c.cu, T]
    kw = dict(window=300, sinks=4)
    first = q.attn_window(c.cache, c.q.cuda(), *args, **kw)
    wide = torch.zeros(c.N, c.Hq + 3, D, dtype=BF, device="cuda")
    wide[:, 2:2 + c.Hq] = c.q.cuda()
    for _ in range(3):
        again = q.attn_window(c.cache, wide[:, 2:2 + c.Hq], *args, **kw)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = q.attn_window(c.cache, wide[:, 2:2 + c.Hq], *args, stream=s, **kw)
    s.synchronize()
    assert torch.equal(first[0], other[0])
    # captured: other lengths and queries at replay, and two graphs with workspaces of their own
    n = q.attn_window_workspace_bytes(c.cache, c.Hq, 2, c.N, T, c.width)
    graphs = []
    for _ in range(2):
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = q.attn_window(c.cache, wide[:, 2:2 + c.Hq], *args, ws=ws, **kw)
        graphs.append((g, out, ws))
    ctx = c.ctx.clone()
    c.ctx.copy_(torch.tensor([700, 30], dtype=torch.int32))
    want = q.attn_window(c.cache, c.q.cuda(), *args, **kw)
    for g, out, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for g, out, _ in graphs:
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    c.ctx.copy_(ctx)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1][0], first[0])


@pytest.mark.parametrize("T,G", [(3, 2), (40, 4)])
def test_missing_pages_and_bad_lengths(T, G):
    """A page that is needed and missing is left out and told; sequences that do not fit, or have
    more tokens than the bound, are left out, their rows as they were."""
    c = Win([50, 40, 20], [T, T, T], 25, 3, 1, G, 64, 16, BF, seed=T)
    hole = (50 - 5) // 16
    c.table[0, hole] = c.k.shape[0] + 5
    c.dev()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full((c.N, c.Hq, 64), 7.0, dtype=BF, device="cuda")
    lse = torch.full((c.N, c.Hq), 7.0, device="cuda")
    ctx = torch.tensor([50, 10 ** 8, 20], dtype=torch.int32, device="cuda")
    q.attn_window(c.cache, c.q.cuda(), c.table.cuda(), ctx, c.cu, T, window=25, sinks=3, o=o, lse=lse, status=st)
    torch.cuda.synchronize()
    assert int(st) == 3
    mid = slice(c.cu_l[1], c.cu_l[2])
    assert torch.all(o[mid] == 7) and torch.all(lse[mid] == 7)
    see = c.seen
    c.seen = lambda b: see(b) & ((torch.arange(see(b).shape[1]) // 16 != hole) | (b != 0))
    rows = c.rows
    c.rows = lambda pool, b, h: torch.where(torch.isfinite(rows(pool, b, h)), rows(pool, b, h), 0.0)
    ref, p = c.reference(0.125), p_rounding(c, 0.125, BF)
    for b in (0, 2):
        sl = slice(c.cu_l[b], c.cu_l[b + 1])
        tol = ref[1][sl] + p[sl] + ref[0][sl].abs() * half_step(BF) + 2.0 ** -24
        assert torch.all((o[sl].double().cpu() - ref[0][sl]).abs() <= tol)
    st.zero_()
    o.fill_(7.0)
    for pool in (c.cache.k, c.cache.v):
        pool.nan_to_num_(0.5)   # (other slots are seen at other lengths)
    cu = torch.tensor([0, T, T + 1, T + 2], dtype=torch.int32, device="cuda")
    q.attn_window(c.cache, c.q.cuda(), c.table.cuda(), ctx * 0 + 20, cu, T - 1, window=25, sinks=3, o=o, lse=lse,
                  status=st)
    torch.cuda.synchronize()
    assert int(st) & 2 and torch.all(o[:T] == 7) and torch.all(o[T + 2:] == 7) and torch.isfinite(o[T:T + 2].float()).all()


def test_nothing_to_do_and_refusals():
    c = Win([20], [4], 9, 0, 1, 2, 64, 16, BF).dev()
    args = (c.q.cuda(), c.table.cuda(), c.ctx, c.cu)
    o, lse = q.attn_window(c.cache, c.q.cuda()[:0], c.table.cuda()[:0], c.ctx[:0], c.cu[:1], 4)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(scale=math.nan)):
        with pytest.raises(q.QmvError):
            q.attn_window(c.cache, *args, 4, **kw)
    for new in (0, -1, 1 << 23):
        with pytest.raises(q.QmvError):
            q.attn_window(c.cache, *args, new)
    with pytest.raises(OverflowError):
        q.attn_window(c.cache, *args, 4, window=1 << 40)
    with pytest.raises(TypeError):
        q.attn_window(c.cache, *args, 4, o_dtype=FP)
    with pytest.raises(TypeError):
        q.attn_window(c.cache, c.q.cuda().float(), *args[1:], 4)
    with pytest.raises(q.QmvError):
        q.attn_window(c.cache, *args, 4, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("T,G,D,dt", [(3, 2, 128, BF), (40, 4, 128, BF), (150, 2, 128, FP), (70, 4, 64, FP),
                                      (150, 2, 64, BF)])
@pytest.mark.parametrize("out", ["same", "fp32"])
@pytest.mark.parametrize("how", ["grow", "leap", "fall"])
def test_scores_that_grow_and_fall_along_the_keys(T, G, D, dt, out, how):
    """Maxima that move at every step, once and late, and never again."""
    c = Win([900], [T], ALL, 0, 2, G, D, 64, dt, seed=T)
    for j in range(900 + T):
        f = {"grow": 2.0 ** (j // 100 - 4), "leap": 24.0 if j == 500 else 0.25, "fall": 2.0 ** (3 - j // 100)}[how]
        c.k[c.table_l[0][j // 64], :, j % 64] *= f
    o, lse = run(c, o_dtype=F32 if out == "fp32" else dt)
    s = D ** -0.5
    check_tree(c, o, lse, c.reference(s), p_rounding(c, s, o.dtype))


@pytest.mark.parametrize("T,D,odt", [(3, 128, BF), (70, 128, BF), (70, 64, F32)])
def test_outputs_on_a_16_byte_boundary_that_is_no_32_byte_one(T, D, odt):
    c = Win([200], [T], 100, 4, 2, 4, D, 16, BF, seed=D)
    o, lse = run(c, o_dtype=odt)
    n = o.numel()
    flat = torch.full((n + 64,), 7.0, dtype=odt, device="cuda")
    at = 16 // flat.element_size()
    odd = flat[at:at + n].view(o.shape)
    assert odd.data_ptr() % 32 == 16
    run(c, o=odd)
    assert torch.equal(odd, o) and torch.all(flat[:at] == 7) and torch.all(flat[at + n:] == 7)


@pytest.mark.parametrize("T,G,D", [(3, 2, 128), (60, 4, 128), (150, 2, 64)])
def test_keys_that_are_not_finite(T, G, D):
    """A NaN key spoils the rows that see it and no others."""
    c = Win([300], [T], 64, 2, 1, G, D, 16, BF, seed=D)
    o, lse = run(c)
    j = 300 + T // 2
    c.k[c.table_l[0][j // 16], :, j % 16, 5] = math.nan
    p, y = run(c)
    see = c.seen(0)[:, j].cuda()
    assert torch.equal(p[~see], o[~see]) and torch.equal(y[~see], lse[~see])
    assert torch.isnan(p[see]).all() and torch.isnan(y[see]).all()
