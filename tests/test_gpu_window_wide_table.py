"""Windows over tables far wider than they, on the GPU: what a call is refused for is its own work,
not the width of the table."""
import pytest

torch = pytest.importorskip("torch")
q = pytest.importorskip("int4_group_quantized_gs64_gb300")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    q.build()
    q.lib()


@pytest.mark.parametrize("T,N", [(1 << 18, 1 << 18), (1, 1), (40, 40)])
def test_width_changes_nothing(T, N):
    g = torch.Generator(device="cuda").manual_seed(T)
    page, pages, Hkv, G, D = 256, 12, 8, 8, 64
    cache = q.AttnCache(*(torch.randn(pages, Hkv, page, D, device="cuda", generator=g, dtype=torch.bfloat16)
                          for _ in range(2)))
    x = torch.randn(N, Hkv * G, D, device="cuda", generator=g, dtype=torch.bfloat16)
    wide = (torch.arange(1 << 22, device="cuda", dtype=torch.int32) * 7 % pages)[None].contiguous()
    narrow = wide[:, :(N + 4000) // page + 2].contiguous()
    ctx = torch.tensor([4000], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    got = []
    for table in (narrow, wide):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got.append(q.attn_window(cache, x, table, ctx, cu, T, window=64, sinks=4, status=st))
        assert int(st) == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert torch.isfinite(got[0][0].float()).all()


def test_overlapping_sequences_that_add_up_to_more_than_a_plan_holds():
    """Each fits, and by N so do all; together (cu goes back to 0 twice) they would be hours of work."""
    N, B, D, page = 1 << 16, 5, 64, 256
    cache = q.AttnCache(*(torch.zeros(2, 8, page, D, device="cuda", dtype=torch.bfloat16) for _ in range(2)))
    x = torch.zeros(N, 64, D, device="cuda", dtype=torch.bfloat16)
    table = torch.zeros(B, 1 << 22, device="cuda", dtype=torch.int32)
    ctx = torch.full((B,), (1 << 30) - N, device="cuda", dtype=torch.int32)
    cu = torch.tensor([0, N, 0, N, 0, N], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = torch.full_like(x, 7.0), torch.full((N, 64), 7.0, device="cuda")
    q.attn_window(cache, x, table, ctx, cu, N, o=o, lse=lse, status=st)
    torch.cuda.synchronize()
    assert int(st) == 2 and torch.all(o == 7) and torch.all(lse == 7)
