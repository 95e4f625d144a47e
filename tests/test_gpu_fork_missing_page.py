"""A fork of a sequence whose last, partly filled page is not there, on the GPU: the child ends with
its whole pages, so that no later call takes a page that was never written for its tokens."""
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


def test_children_end_before_a_page_that_is_not_there():
    table = [[0, 1, -1, -1], [2, -5, -1, -1], [99, -1, -1, -1], [3, 4, -1, -1], [-1, 5, -1, -1]]
    lens = [20, 20, 7, 32, 20]             # there; none; past the pool; whole pages only; a hole before the last
    refs, st = i32([1] * 6 + [0] * 6), i32([0])
    t, n, m = q.attn_pages_fork(refs, i32(table), i32(lens), i32([0, 1, 2, 3, 4, 1]), 16, status=st)
    assert int(st) == 1
    assert n.tolist() == [20, 16, 0, 32, 20, 16]
    assert t.tolist() == [[0, 6, -1, -1], [2, -1, -1, -1], [-1] * 4, [3, 4, -1, -1], [-1, 7, -1, -1], [2, -1, -1, -1]]
    assert m.tolist() == [[1, 6, 4], [-1, -1, 0], [-1, -1, 0], [-1, -1, 0], [5, 7, 4], [-1, -1, 0]]
    assert refs.tolist() == [2, 1, 3, 2, 2, 1, 1, 1] + [0] * 4


def test_the_next_update_takes_no_page_for_tokens_that_were_not_copied():
    refs, st = i32([1, 0, 0, 0]), i32([0])
    t, n, _ = q.attn_pages_fork(refs, i32([[0, -1, -1]]), i32([20]), i32([0]), 16, status=st)
    q.attn_pages_update(refs, t, n, i32([0]), 16)
    assert int(st) == 1 and t.tolist() == [[0, -1, -1]] and refs.tolist() == [2, 0, 0, 0]
