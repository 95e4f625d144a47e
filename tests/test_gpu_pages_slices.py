"""Forks, compaction and updates with outputs that are slices of one buffer, on the GPU: neighbours
are taken, slices that overlap are refused and nothing is written."""
import pytest

torch = pytest.importorskip("torch")
q = pytest.importorskip("int4_group_quantized_gs64_gb300")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    q.build()
    q.lib()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_fork_into_the_rows_behind_its_parents():
    """One buffer of tables, one of everything of a row: parents, children, lengths, moves."""
    rows, flat = torch.full((8, 3), -1, dtype=torch.int32, device="cuda"), torch.full((40,), -9, dtype=torch.int32, device="cuda")
    rows[:2] = i32([[0, 1, -1], [2, -1, -1]])
    refs, lens, parent, new_lens, moves = (flat[a:b] for a, b in ((0, 10), (10, 12), (12, 17), (17, 22), (22, 37)))
    refs.copy_(i32([1, 1, 1] + [0] * 7)), lens.copy_(i32([20, 16])), parent.copy_(i32([0, 1, 1, 0, 1]))
    moves = moves.view(5, 3)
    t, n, m = q.attn_pages_fork(refs, rows[:2], lens, parent, 16, new_table=rows[2:7], new_lens=new_lens, moves=moves)
    none = [-1, -1, 0]
    assert rows.tolist() == [[0, 1, -1], [2, -1, -1], [0, 3, -1], [2, -1, -1], [2, -1, -1], [0, 4, -1], [2, -1, -1], [-1] * 3]
    assert n.tolist() == [20, 16, 16, 20, 16] and m.tolist() == [[1, 3, 4], none, none, [1, 4, 4], none]
    assert refs.tolist() == [3, 1, 4, 1, 1] + [0] * 5 and flat[37:].tolist() == [-9] * 3
    before = rows.clone(), flat.clone()
    kw = dict(new_table=rows[2:7], new_lens=new_lens, moves=moves)
    for bad in (dict(new_table=rows[1:6]), dict(new_lens=flat[16:21]), dict(new_lens=flat[11:16]), dict(new_lens=flat[18:23]),
                dict(moves=flat[11:26].view(5, 3)), dict(moves=flat[20:35].view(5, 3)), dict(new_table=flat[9:24].view(5, 3))):
        with pytest.raises(q.QmvError):
            q.attn_pages_fork(refs, rows[:2], lens, parent, 16, **{**kw, **bad})
    torch.cuda.synchronize()
    assert torch.equal(rows, before[0]) and torch.equal(flat, before[1])


def test_compact_and_update():
    cache = q.AttnCache.empty(4, 1, 16, 64)
    cache.k.normal_(), cache.v.normal_()
    flat = i32([0, 1, 2, 3, 5, 9, 0, 4, 6, 2, 1, 1, 3, 0, 2, 1, -7, -7, -7])
    table, ctx, cu, kept, keep, new = (flat[a:b] for a, b in ((0, 4), (4, 6), (6, 9), (9, 11), (11, 17), (17, 19)))
    table = table.view(2, 2)
    k = cache.k.clone()
    out = q.attn_compact(cache, table, ctx, cu, keep[:6], kept, new_ctx=new)
    assert out.tolist() == [7, 10] and flat[:17].tolist() == [0, 1, 2, 3, 5, 9, 0, 4, 6, 2, 1, 1, 3, 0, 2, 1, -7]
    assert torch.equal(cache.k[0, 0, 5], k[0, 0, 6]) and torch.equal(cache.k[0, 0, 6], k[0, 0, 8])
    assert torch.equal(cache.k[2, 0, 9], k[2, 0, 10])
    before = flat.clone(), cache.k.clone()
    for a in (0, 3, 4, 5, 8, 10, 12, 16):
        with pytest.raises(q.QmvError):
            q.attn_compact(cache, table, ctx, cu, keep, kept, new_ctx=flat[a:a + 2])
    refs, lens = i32([1] * 4), ctx
    for bad in (dict(table=flat[1:5].view(2, 2)), dict(refs=flat[5:9]), dict(refs=flat[2:6]), dict(more=flat[3:5])):
        with pytest.raises(q.QmvError):
            q.attn_pages_update(**{**dict(refs=refs, table=table, lens=lens, more=lens, page=16), **bad})
    torch.cuda.synchronize()
    assert torch.equal(flat, before[0]) and torch.equal(cache.k, before[1]) and refs.tolist() == [1] * 4
    q.attn_pages_update(refs, table, lens, lens, 16)     # lengths and tokens to come may be one array
    assert table.tolist() == [[0, -1], [2, 3]] and refs.tolist() == [1, 0, 1, 1]
