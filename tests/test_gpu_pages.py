"""The upkeep of a cache's pages on the GPU against plain lists: whole numbers, so equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
q = pytest.importorskip("int4_group_quantized_gs64_gb300")

pytestmark = pytest.mark.gpu
ALL = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    q.build()
    q.lib()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


class Pool:
    """refs and a table as plain lists, with the rules of the calls."""

    def __init__(self, pages, B, width, page):
        self.refs, self.page = [0] * pages, page
        self.table = [[-1] * width for _ in range(B)]

    def needs(self, i, n, more, W, S):
        a, b = i * self.page, (i + 1) * self.page
        return a < n + more and (a < S or b > n - W + 1)

    def update(self, lens, more, W, S):
        """Returns the status."""
        st, width = 0, len(self.table[0])
        ok = [n >= 0 and m >= 0 and n + m <= width * self.page for n, m in zip(lens, more)]
        st |= 0 if all(ok) else 2
        for b, row in enumerate(self.table):
            for i, x in enumerate(row):
                if x >= len(self.refs):
                    st |= 1
                elif ok[b] and x >= 0 and not self.needs(i, lens[b], more[b], W, S):
                    if self.refs[x] <= 0:
                        st |= 1
                    else:
                        self.refs[x] -= 1
                    row[i] = -1
        free = [p for p, r in enumerate(self.refs) if r == 0][::-1]
        for b, row in enumerate(self.table):
            for i, x in enumerate(row):
                if ok[b] and x < 0 and self.needs(i, lens[b], more[b], W, S):
                    if free:
                        row[i] = free.pop()
                        self.refs[row[i]] = 1
                    else:
                        st |= 8
        return st

    def fork(self, lens, parent):
        new, new_lens, moves, st = [], [], [], 0
        width = len(self.table[0])
        for p in parent:
            n = lens[p] if 0 <= p < len(lens) else -1
            row, mv = [-1] * width, [-1, -1, 0]
            if 0 <= n <= width * self.page:
                w, r = divmod(n, self.page)
                for i in range(w):
                    x = self.table[p][i]
                    st |= x >= len(self.refs)
                    if 0 <= x < len(self.refs):
                        row[i] = x
                        self.refs[x] += 1
                if r:
                    x = self.table[p][w]
                    if 0 <= x < len(self.refs):
                        mv = [x, -1, r]
                    else:
                        st |= 1
            else:
                st, n = st | 2, 0
            new.append(row), new_lens.append(n), moves.append(mv)
        free = [p for p, r in enumerate(self.refs) if r == 0][::-1]
        for f, mv in enumerate(moves):
            if mv[2] == 0:
                continue
            if free:
                mv[1] = free.pop()
                self.refs[mv[1]] = 1
                new[f][new_lens[f] // self.page] = mv[1]
            else:
                st |= 8
                new_lens[f] -= new_lens[f] % self.page
                moves[f] = [-1, -1, 0]
        return new, new_lens, moves, st


@pytest.mark.parametrize("pages,B,width,page,W,S", [
    (10, 1, 4, 16, ALL, 0), (40, 3, 9, 16, 20, 0), (40, 3, 9, 16, 20, 17), (300, 40, 20, 64, 100, 4),
    (300, 7, 700, 16, 1, 130), (9000, 5, 1500, 16, ALL, 0), (5000, 500, 30, 32, 200, 1), (20, 6, 9, 256, 300, 4)])
def test_update_follows_its_rules_over_steps(pages, B, width, page, W, S):
    """Drawn lengths that grow, are cut back and end; pools that run out of pages among them."""
    rng = np.random.default_rng(pages + B)
    pool = Pool(pages, B, width, page)
    refs, table = i32(pool.refs), i32(pool.table)
    lens, st = np.zeros(B, int), status()
    ws = torch.empty(q.attn_pages_update_workspace_bytes(pages, B, width), dtype=torch.uint8, device="cuda")
    seen = 0
    for step in range(12):
        kind = rng.integers(0, 6, B)
        lens = np.where(kind == 0, 0, np.where(kind == 1, lens // 2, np.minimum(
            lens + rng.integers(0, 2 * page + 2 * W % 977, B), width * page)))
        more = np.where(kind == 0, 0, np.minimum(rng.integers(0, 3 * page, B), width * page - lens))
        want = pool.update(lens.tolist(), more.tolist(), W, S)
        st.zero_()
        q.attn_pages_update(refs, table, i32(lens), i32(more), page, window=W, sinks=S, ws=ws, status=st)
        assert table.tolist() == pool.table and refs.tolist() == pool.refs and int(st) == want, step
        seen |= want
        lens = np.where(kind == 0, 0, lens + more)
    q.attn_pages_update(refs, table, i32([0] * B), i32([0] * B), page)
    assert not refs.any() and torch.all(table == -1)


def test_update_many_pages_to_find():
    """More free pages asked for than one look at refs finds, most of the pool held."""
    rng = np.random.default_rng(1)
    pages, B, width = 100003, 60, 900
    pool = Pool(pages, B, width, 16)
    pool.refs = (rng.random(pages) < 0.6).astype(int).tolist()
    refs, table, st = i32(pool.refs), i32(pool.table), status()
    more = rng.integers(0, width * 16 + 1, B).tolist()
    want = pool.update([0] * B, more, ALL, 0)
    q.attn_pages_update(refs, table, i32([0] * B), i32(more), 16, status=st)
    assert table.tolist() == pool.table and refs.tolist() == pool.refs and int(st) == want
    assert sum(x >= 0 for row in pool.table for x in row) > 8192


def test_update_bad_rows_are_left_alone():
    pool = Pool(6, 5, 4, 16)
    pool.table = [[0, 1, -1, -1], [2, 99, -9, -1], [3, 3, -1, -1], [4, -1, -1, -1], [5, -1, -1, -1]]
    pool.refs = [1, 1, 1, 1, 1, 0]        # page 3 is held twice, page 5 by nobody, says refs
    refs, table, st = i32(pool.refs), i32(pool.table), status()
    lens, more = [-1, 16, 0, 60, 0], [0, 16, 0, 5, 0]
    want = pool.update(lens, more, ALL, 0)
    q.attn_pages_update(refs, table, i32(lens), i32(more), 16, status=st)
    assert table.tolist() == pool.table and refs.tolist() == pool.refs
    assert int(st) == want == 3
    assert pool.table[0] == [0, 1, -1, -1] and pool.table[3] == [4, -1, -1, -1] and pool.table[1][1] == 99


@pytest.mark.parametrize("pages,B,width,page,F", [(8, 1, 3, 16, 1), (40, 3, 9, 16, 11), (3000, 64, 71, 128, 256),
                                                  (20000, 5, 1500, 16, 9), (6000, 33, 12, 32, 2500)])
def test_fork_follows_its_rules(pages, B, width, page, F):
    rng = np.random.default_rng(F)
    pool = Pool(pages, B, width, page)
    lens = rng.integers(0, width * page + 1, B)
    lens[0] = width * page - page             # whole pages only
    if B > 2:
        lens[1:3] = 0, page - 1
    lens = lens.tolist()
    refs, table, st = i32(pool.refs), i32(pool.table), status()
    assert pool.update(lens, [0] * B, ALL, 0) in (0, 8)
    q.attn_pages_update(refs, table, i32(lens), i32([0] * B), page)
    for _ in range(2):                        # the second time from pages that are shared already
        parent = rng.integers(0, B, F).tolist()
        new, new_lens, moves, want = pool.fork(lens, parent)
        st.zero_()
        t, n, m = q.attn_pages_fork(refs, table, i32(lens), i32(parent), page, status=st)
        assert t.tolist() == new and n.tolist() == new_lens and m.tolist() == moves and int(st) == want
        assert refs.tolist() == pool.refs


def test_fork_bad_parents_and_lengths():
    pool = Pool(10, 3, 4, 16)
    pool.table = [[0, 1, -1, -1], [2, 77, 3, -1], [4, -1, -1, -1]]
    pool.refs = [1, 1, 1, 1, 1] + [0] * 5
    lens, parent = [20, 64, -3], [0, 1, 2, 3, -1, 0]
    refs, st = i32(pool.refs), status()
    new, new_lens, moves, want = pool.fork(lens, parent)
    t, n, m = q.attn_pages_fork(refs, i32(pool.table), i32(lens), i32(parent), 16, status=st)
    assert t.tolist() == new and n.tolist() == new_lens and m.tolist() == moves and int(st) == want == 3
    assert refs.tolist() == pool.refs


@pytest.mark.parametrize("D,page,Hkv,dt", [(64, 16, 1, torch.bfloat16), (128, 128, 8, torch.float16),
                                           (128, 256, 3, torch.bfloat16)])
def test_copy(D, page, Hkv, dt):
    g = torch.Generator().manual_seed(page)
    k, v = (torch.randn(9, Hkv, page, D, generator=g).to(dt) for _ in range(2))
    dk, dv = (torch.randn(12, Hkv, page, D, generator=g).to(dt) for _ in range(2))
    acc, dacc = torch.rand(9, Hkv, page, generator=g), torch.rand(12, Hkv, page, generator=g)
    moves = [[0, 11, page], [3, 2, 1], [-1, -1, 0], [8, 0, page - 1], [1, 5, 0], [-1, 4, 7], [3, 7, 5], [2, -2, 3]]
    src, dst, st = q.AttnCache(k.cuda(), v.cuda()), q.AttnCache(dk.cuda(), dv.cuda()), status()
    out = dacc.cuda()
    q.attn_pages_copy(src, dst, i32(moves), src_acc=acc.cuda(), dst_acc=out, status=st)
    for s, d, n in moves:
        if s >= 0 and d >= 0:
            for a, b in ((k, dk), (v, dv), (acc, dacc)):
                b[d, :, :n] = a[s, :, :n]
    assert int(st) == 0
    assert torch.equal(dst.k.cpu(), dk) and torch.equal(dst.v.cpu(), dv) and torch.equal(out.cpu(), dacc)
    assert torch.equal(src.k.cpu(), k) and torch.equal(src.v.cpu(), v)
    # within one cache, weights cleared; what does not fit is left out and told
    own = acc.cuda()
    q.attn_pages_copy(src, src, i32([[0, 8, 3], [9, 1, 2], [1, 9, 2], [1, 2, page + 1], [1, 2, -1]]), dst_acc=own, status=st)
    k[8, :, :3], v[8, :, :3], acc[8, :, :3] = k[0, :, :3], v[0, :, :3], 0
    assert int(st) == 3
    assert torch.equal(src.k.cpu(), k) and torch.equal(src.v.cpu(), v) and torch.equal(own.cpu(), acc)
    q.attn_pages_copy(src, dst, i32([]).view(0, 3))


def compact_reference(pools, table, page, ctx, cu, keep, kept):
    for b in range(len(ctx)):
        src = [ctx[b] + keep[cu[b] + i] for i in range(kept[b])]
        for pool in pools:
            rows = [pool[table[b][s // page], :, s % page].clone() for s in src]
            for i, r in enumerate(rows):
                s = ctx[b] + i
                pool[table[b][s // page], :, s % page] = r


@pytest.mark.parametrize("D,page,Hkv,T,B", [(64, 16, 2, 7, 3), (128, 64, 8, 61, 5), (128, 16, 1, 700, 2),
                                            (64, 256, 3, 300, 4), (64, 16, 1, 4, 900)])
def test_compact(D, page, Hkv, T, B):
    rng = np.random.default_rng(T)
    g = torch.Generator().manual_seed(T)
    drafts = rng.integers(0, T + 1, B)
    drafts[0] = T
    ctx = rng.integers(0, 100, B).tolist()
    cu = [0] + np.cumsum(drafts).tolist()
    width = -(-(100 + T) // page)
    table = rng.permutation(B * width + 2)[:B * width].reshape(B, width).tolist()
    keep, kept = np.full(cu[-1], 10 ** 6), []
    for b, t in enumerate(drafts):
        n = int(rng.integers(0, t + 1)) if b % 3 else t - (t > 1)
        keep[cu[b]:cu[b] + n] = np.sort(rng.choice(t, n, replace=False)) if t else []
        kept.append(n)
    if B > 1:
        kept[1] = int(drafts[1])             # one that keeps all
        keep[cu[1]:cu[2]] = np.arange(drafts[1])
    k, v = (torch.randn(B * width + 2, Hkv, page, D, generator=g).to(torch.bfloat16) for _ in range(2))
    acc = torch.rand(B * width + 2, Hkv, page, generator=g)
    cache, a, st = q.AttnCache(k.cuda(), v.cuda()), acc.cuda(), status()
    out = q.attn_compact(cache, i32(table), i32(ctx), i32(cu), i32(keep), i32(kept), acc=a, status=st)
    compact_reference((k, v, acc), table, page, ctx, cu, keep.tolist(), kept)
    assert int(st) == 0 and out.tolist() == [c + n for c, n in zip(ctx, kept)]
    assert torch.equal(cache.k.cpu(), k) and torch.equal(cache.v.cpu(), v) and torch.equal(a.cpu(), acc)


def test_compact_refuses_and_leaves_out():
    """Tokens out of order, twice, or not the sequence's: nothing of it moves."""
    g = torch.Generator().manual_seed(0)
    k = torch.randn(20, 1, 16, 64, generator=g).to(torch.float16)
    cache, st = q.AttnCache(k.cuda(), k.cuda()), status()
    table = [[2 * b, 2 * b + 1] for b in range(8)] + [[16, 25]]
    keep = [1, 0, 3, 3, 1, 4, -1, 2, 1, 3, 2, 3, 0, 2, 1, 3, 1, 15]
    cu = [0, 2, 4, 6, 8, 10, 12, 14, 16, 18]
    kept = [2, 2, 2, 2, 3, -1, 1, 1, 2]      # order, twice and past, past, negative, too many, negative; fine; fine; past
    ctx = [5] * 6 + [15, 31, 5]              # the eighth: its drafts do not fit the table
    out = q.attn_compact(cache, i32(table), i32(ctx), i32(cu), i32(keep), i32(kept), status=st)
    torch.cuda.synchronize()
    assert int(st) == 2 and out.tolist() == ctx[:6] + [16, 31, 5]
    assert torch.equal(cache.k.cpu(), k)     # (the seventh keeps what is in its place)
    # a page that is missing: the other rows move
    st.zero_()
    keep, kept = [1, 3, 5, 0, 0, 0], [3]
    out = q.attn_compact(cache, i32([[4, 99]]), i32([13]), i32([0, 6]), i32(keep), i32(kept), status=st)
    torch.cuda.synchronize()
    want = k.clone()
    want[4, :, 13] = k[4, :, 14]
    assert int(st) == 1 and out.tolist() == [16] and torch.equal(cache.k.cpu(), want)


def test_streams_graphs_and_refusals():
    pool = Pool(64, 4, 8, 16)
    refs, table, st = i32(pool.refs), i32(pool.table), status()
    lens, more = i32([10, 0, 40, 7]), i32([8, 0, 8, 100])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q.attn_pages_update(refs, table, lens, more, 16, stream=s)
    t, n, m = q.attn_pages_fork(refs, table, lens, i32([2, 0]), 16, stream=s)
    s.synchronize()
    pool.update(lens.tolist(), more.tolist(), ALL, 0)
    new, new_lens, moves, _ = pool.fork(lens.tolist(), [2, 0])
    assert table.tolist() == pool.table and (t.tolist(), n.tolist(), m.tolist()) == (new, new_lens, moves)
    # captured: other lengths at replay
    parent = i32([0, 3, 3])
    ws = [torch.empty(x, dtype=torch.uint8, device="cuda") for x in (
        q.attn_pages_update_workspace_bytes(64, 4, 8), q.attn_pages_fork_workspace_bytes(64, 3))]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.attn_pages_update(refs, table, lens, more, 16, window=30, sinks=4, ws=ws[0], status=st)
        t, n, m = q.attn_pages_fork(refs, table, lens, parent, 16, ws=ws[1], status=st)
    for a, b in (([60, 3, 41, 100], [3, 40, 1, 20]), ([61, 4, 0, 128], [1, 1, 0, 0])):
        lens.copy_(i32(a)), more.copy_(i32(b))
        g.replay()
        want = pool.update(a, b, 30, 4)
        new, new_lens, moves, w2 = pool.fork(a, [0, 3, 3])
        assert int(st) == want | w2 and table.tolist() == pool.table and refs.tolist() == pool.refs
        assert (t.tolist(), n.tolist(), m.tolist()) == (new, new_lens, moves)
        st.zero_()
    for bad in (dict(page=24), dict(window=0), dict(sinks=-1)):
        with pytest.raises(q.QmvError):
            q.attn_pages_update(refs, table, lens, more, **{"page": 16, **bad})
    with pytest.raises((TypeError, ValueError)):
        q.attn_pages_update(refs, table, lens[:3], more, 16)
    with pytest.raises((TypeError, ValueError)):
        q.attn_pages_update(refs.cpu(), table, lens, more, 16)
    with pytest.raises(q.QmvError):
        q.attn_pages_fork(refs, table, lens, i32([0, 1, 2, 3]), 16, new_table=table)
    c = q.AttnCache.empty(4, 1, 16, 64)
    with pytest.raises(ValueError):
        q.attn_pages_copy(c, c, i32([0, 1, 2]))
    with pytest.raises(q.QmvError):
        q.attn_pages_copy(c, q.AttnCache.empty(4, 2, 16, 64), i32([[0, 1, 2]]))
    ctx = i32([1])
    with pytest.raises(q.QmvError):
        q.attn_compact(c, i32([[0]]), ctx, i32([0, 1]), i32([0]), i32([1]), new_ctx=ctx)
