"""Normed rotary append on the GPU against a plain 64-bit form.

A normed element x w r is off by at most 20 * 2^-24 of itself: the squares of a head
are added up in at most 20 fp32 steps, which the root halves (10), eps is added (1/2),
rsqrtf is off by 2 steps of 2^-23 (4), and two products follow (2). The turn and the
rounding to the cache's type are bounded as without norms."""
import math

import pytest

torch = pytest.importorskip("torch")
q = pytest.importorskip("int4_group_quantized_gs64_gb300")

from test_gpu_attn import BF, FP, F32, Case, half_step, rope_reference  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    q.build()
    q.lib()


def normed(x, w, eps):
    x = x.double()
    r = (x.square().mean(-1, keepdim=True) + eps)
    r = torch.where(r == 0, 0.0, r ** -0.5)
    return x * r * (1.0 if w is None else w.double())


def reference(x, w, eps, pos, inv, rot, inter, m, dt):
    """The heads' values and their bounds, for heads that share the weights w."""
    y = normed(x, w, eps)
    rel = 20 * 2.0 ** -24
    e = y.abs() * rel
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    pair = (e[..., i] + e[..., j]) * abs(m)
    e[..., i], e[..., j] = pair, pair
    z, turn = rope_reference(y, pos, inv, rot, inter, m)
    return z, e + turn.abs() + z.abs() * half_step(dt) + 2.0 ** -25


CASES = [
    # ctx, drafts, Hkv, G, D, page, cache, input, weights, rot, interleaved
    ([0], [1], 1, 1, 64, 16, BF, BF, F32, 64, False),
    ([5000], [1], 8, 6, 128, 64, BF, BF, BF, 128, False),
    ([7, 0, 250], [3, 0, 70], 2, 3, 128, 16, FP, F32, FP, 64, True),
    ([100000, 31], [5, 2], 2, 2, 64, 32, BF, F32, F32, 32, False),
    ([15, 16], [17, 300], 1, 4, 128, 128, FP, FP, F32, 128, True),
    ([3], [900], 1, 5, 64, 16, FP, FP, None, 64, False),
    ([3], [9], 2, 2, 64, 16, FP, F32, F32, 50, False),       # rot no multiple of 16
    ([3], [9], 2, 2, 64, 16, BF, BF, BF, 6, True),
    ([3], [9], 3, 1, 128, 16, BF, BF, None, 2, False),
]


def inputs(c, src, wt, rot, seed=1, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(c.N, c.Hq + 2 * c.Hkv, c.D, generator=g) * scale).to(src)
    w = [None if wt is None else (1 + 0.5 * torch.randn(c.D, generator=g)).to(wt) for _ in range(2)]
    pos = torch.randint(0, 1 << 20, (c.N,), generator=g, dtype=torch.int32)
    inv = torch.tensor([10000.0 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    return qkv, w, pos, inv


def call(c, qkv, w, pos, inv, **kw):
    d = qkv.cuda()
    return q.attn_norm_rope_append(c.cache, d[:, :c.Hq], d[:, c.Hq:c.Hq + c.Hkv], d[:, c.Hq + c.Hkv:],
                                   *(None if x is None else x.cuda() for x in w), pos.cuda(), inv.cuda(),
                                   c.table.cuda(), c.ctx, c.cu, **kw)


def check(c, out, qkv, w, pos, inv, rot, inter, m, eps, acc=None):
    y, tol = reference(qkv[:, :c.Hq], w[0], eps, pos, inv, rot, inter, m, c.dtype)
    assert torch.all((out.double().cpu() - y).abs() <= tol), float(((out.double().cpu() - y).abs() / tol).max())
    y, tol = reference(qkv[:, c.Hq:c.Hq + c.Hkv], w[1], eps, pos, inv, rot, inter, m, c.dtype)
    k, v = c.cache.k.cpu(), c.cache.v.cpu()
    new = torch.zeros(k.shape[0], c.page, dtype=torch.bool)
    for b in range(c.B):
        for t in range(c.drafts[b]):
            s, n = c.ctx_l[b] + t, c.cu_l[b] + t
            pg, rw = c.table_l[b][s // c.page], s % c.page
            assert torch.all((k[pg, :, rw].double() - y[n]).abs() <= tol[n])
            assert torch.equal(v[pg, :, rw], qkv[n, c.Hq + c.Hkv:].to(c.dtype))
            new[pg, rw] = True
    old = ~new[:, None, :].expand(-1, c.Hkv, -1)
    assert torch.equal(k[old], c.k[old]) and torch.equal(v[old], c.v[old])
    if acc is not None:
        a = acc.cpu()
        assert torch.equal(a[old], c.acc[old]) and not a[~old].any()


@pytest.mark.parametrize("shape", CASES, ids=[str(i) for i in range(len(CASES))])
def test_norm_rope_append(shape):
    ctx, drafts, Hkv, G, D, page, dt, src, wt, rot, inter = shape
    c = Case(ctx, drafts, Hkv, G, D, page, dt, seed=rot).dev()
    qkv, w, pos, inv = inputs(c, src, wt, rot)
    m, eps = (1.25, 1e-5) if inter else (1.0, 0.5)
    acc = c.acc.cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(c, qkv, w, pos, inv, eps=eps, interleaved=inter, mscale=m, acc=acc, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0 and out.dtype == dt
    check(c, out, qkv, w, pos, inv, rot, inter, m, eps, acc)


@pytest.mark.parametrize("rot", [64, 6])
def test_small_large_and_zero_heads(rot):
    """Heads of zeros stay zeros with eps = 0; magnitudes far from one come out of size one."""
    c = Case([10], [12], 2, 2, 64, 16, BF, seed=1).dev()
    qkv, w, pos, inv = inputs(c, F32, F32, rot)
    qkv[0], qkv[1], qkv[2] = 0.0, qkv[1] * 1e-12, qkv[2] * 1e12
    out = call(c, qkv, w, pos, inv, eps=0.0)
    torch.cuda.synchronize()
    assert not out[0].any()
    check(c, out, qkv, w, pos, inv, rot, False, 1.0, 0.0)
    out = call(c, qkv, w, pos, inv, eps=1e-6)
    check(c, out, qkv, w, pos, inv, rot, False, 1.0, 1e-6)


def test_one_weight_and_unaligned_ones():
    """A weight that is left out counts as ones; weights off 16-byte boundaries."""
    c = Case([20], [11], 2, 3, 128, 16, FP, seed=2).dev()
    qkv, w, pos, inv = inputs(c, FP, F32, 128)
    for pair in ((w[0], None), (None, w[1])):
        out = call(c, qkv, pair, pos, inv)
        check(c, out, qkv, pair, pos, inv, 128, False, 1.0, 1e-6)
    d = qkv.cuda()
    flat = [torch.cat([torch.zeros(1), x]).cuda()[1:] for x in w]
    out = q.attn_norm_rope_append(c.cache, d[:, :c.Hq], d[:, c.Hq:c.Hq + 2], d[:, c.Hq + 2:], *flat, pos.cuda(),
                                  inv.cuda(), c.table.cuda(), c.ctx, c.cu)
    torch.cuda.synchronize()
    check(c, out, qkv, w, pos, inv, 128, False, 1.0, 1e-6)


def test_stream_graph_and_same_bits():
    c = Case([20, 3], [5, 40], 2, 4, 128, 16, BF, seed=3).dev()
    qkv, w, pos, inv = inputs(c, BF, BF, 128)
    first = call(c, qkv, w, pos, inv)
    torch.cuda.synchronize()
    k0 = c.cache.k.clone()
    d, wd = qkv.cuda(), [x.cuda() for x in w]
    args = (c.cache, d[:, :c.Hq], d[:, c.Hq:c.Hq + 2], d[:, c.Hq + 2:], *wd, pos.cuda(), inv.cuda(), c.table.cuda(),
            c.ctx, c.cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = q.attn_norm_rope_append(*args, stream=s)
    s.synchronize()
    assert torch.equal(out, first)
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = q.attn_norm_rope_append(*args)
    c.cache.k.zero_()
    d.mul_(-1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -first)
    new = c.cache.k != 0
    assert torch.equal(c.cache.k[new], -k0[new]) and new.flatten(1).any(1).any()


def test_bad_pages_and_lengths():
    c = Case([20, 8], [4, 4], 1, 2, 64, 16, BF, seed=0).dev()
    qkv, w, pos, inv = inputs(c, BF, BF, 64)
    c.table[0, 1] = -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(c, qkv, w, pos, inv, status=st)
    torch.cuda.synchronize()
    changed = (c.cache.k.cpu() != c.k).flatten(1).any(1).nonzero().flatten().tolist()
    assert int(st) == 1 and changed == [c.table_l[1][0]] and torch.isfinite(out.float()).all()


def test_refusals():
    c = Case([20], [4], 2, 2, 64, 16, BF, seed=0).dev()
    qkv, w, pos, inv = inputs(c, BF, F32, 64)
    for bad in ((w[0][:63], w[1]), (w[0].half(), w[1]), (w[0], w[1].to(BF)), (w[0].double(), w[1].double())):
        with pytest.raises((TypeError, ValueError)):
            call(c, qkv, bad, pos, inv)
    for eps in (-1e-6, math.inf, math.nan):
        with pytest.raises(q.QmvError):
            call(c, qkv, w, pos, inv, eps=eps)
    with pytest.raises(ValueError):
        call(c, qkv, (w[0].cuda(), w[1].cuda().repeat(2)[::2]), pos, inv)      # not contiguous
    torch.cuda.synchronize()
    assert torch.equal(c.cache.k.cpu(), c.k)


@pytest.mark.parametrize("Hkv,G,D,src", [(2, 6, 128, BF), (2, 7, 128, BF), (8, 5, 128, F32), (2, 14, 64, F32),
                                         (2, 15, 64, BF), (8, 8, 64, BF), (1, 1, 128, F32)])
def test_few_and_many_heads(Hkv, G, D, src):
    """Up to four passes of a warp over a token's heads, and more; the last pass full or not."""
    c = Case([33, 0, 700], [5, 1, 130], Hkv, G, D, 32, BF, seed=G).dev()
    qkv, w, pos, inv = inputs(c, src, F32, D // 2)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(c, qkv, w, pos, inv, eps=1e-5, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    check(c, out, qkv, w, pos, inv, D // 2, False, 1.0, 1e-5)
