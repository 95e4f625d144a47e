"""The forms of windowed attention on the GPU, each with the values and masks where it can go wrong:
up to 16 rows a key/value head, up to 128 (one tile, whose two streams take alternate steps and are
added up at the end), and more (two tiles). Bounds as in test_gpu_window."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
q = pytest.importorskip("int4_group_quantized_gs64_gb300")

from test_gpu_attn import BF, FP, F32, check_tree, half_step, p_rounding  # noqa: E402
from test_gpu_window import ALL, Win, run  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    q.build()
    q.lib()


def form(T, G):
    """What set_rows picks."""
    if T * G <= 16:
        return "rows"
    return "one" if G <= 128 and T <= 128 // G else "two"


# new tokens, query heads a key/value head, elements a head, type
ONE = [(20, 4, 128, BF), (9, 6, 128, FP), (60, 2, 64, BF), (32, 4, 64, FP), (100, 1, 128, BF), (2, 60, 64, BF), (1, 128, 128, FP)]
TWO = [(33, 4, 128, BF), (150, 2, 128, FP), (150, 1, 64, BF), (3, 50, 64, FP)]
FEW = [(3, 4, 128, BF), (4, 4, 128, FP)]
FORMS = [("one",) + x for x in ONE] + [("two",) + x for x in TWO] + [("rows",) + x for x in FEW]
IDS = ["-".join(map(str, f[:4])) + ("-bf16" if f[4] is BF else "-fp16") for f in FORMS]
every_form = pytest.mark.parametrize("what,T,G,D,dt", FORMS, ids=IDS)
both_outputs = pytest.mark.parametrize("out", ["same", "fp32"])


def odt(dt, out):
    return F32 if out == "fp32" else dt


def test_the_forms_are_what_they_are_called():
    assert all(form(T, G) == what for what, T, G, _, _ in FORMS)


@every_form
@both_outputs
@pytest.mark.parametrize("ctx,W,S", [(50, 20, 3), (2900, 1700, 40), (700, ALL, 0)])
def test_infinities_of_values_reach_those_that_see_them(what, T, G, D, dt, out, ctx, W, S):
    """At the first tokens, the window's edge and the diagonal, in both halves of a head; items of one
    block and of many."""
    c = Win([ctx, 7], [T, T], W, S, 1, G, D, 16, dt, seed=T)
    clean = c.v.clone()
    edge = max(0, ctx - W + 2)
    marks = [(0, edge, math.nan, 1), (0, ctx + T // 2, -math.inf, D - 1), (0, ctx, math.inf, D // 2 - 1), (1, 8, math.inf, D // 2 + 3)]
    if S:
        marks.append((0, S - 1, math.inf, 5))
    if W < ALL:
        marks.append((0, edge + max(0, T // 2 - 2), math.inf, D // 2))
    hit = torch.zeros(c.N, D, dtype=torch.bool)
    for b, j, x, e in marks:
        if j >= c.ctx_l[b] + T:
            continue
        pg, rw = c.table_l[b][j // 16], j % 16
        if pg < 0:
            continue
        c.v[pg, :, rw, e] = x
        clean[pg, :, rw, e] = 0
        hit[c.cu_l[b]:c.cu_l[b + 1], e] |= c.seen(b)[:, j]
    o, lse = run(c, o_dtype=odt(dt, out))
    o = o.cpu()
    hit = hit[:, None].expand(-1, c.Hq, -1)
    assert not torch.isfinite(o[hit]).any() and torch.isfinite(o[~hit]).all()
    c.v = clean
    ref, s = c.reference(D ** -0.5), D ** -0.5
    o[hit] = ref[0][hit].to(o.dtype)
    check_tree(c, o, lse, ref, p_rounding(c, s, o.dtype))


@every_form
@both_outputs
def test_rows_of_scores_minus_inf(what, T, G, D, dt, out):
    """All keys that a sequence sees score -inf: zeros, also over infinite values; the other's are as they were."""
    c = Win([40, 25, 300], [T, T, T], 30, 2, 2, G, D, 16, dt, seed=T, qscale=1.0)
    c.q[c.cu_l[1]:c.cu_l[2]] = c.q[c.cu_l[1]:c.cu_l[2]].abs() + 0.5
    for j in range(25 + T):
        if c.table_l[1][j // 16] >= 0:
            c.k[c.table_l[1][j // 16], :, j % 16] = -math.inf
    c.v[c.table_l[1][25 // 16], :, 25 % 16, 3] = math.inf
    o, lse = run(c, o_dtype=odt(dt, out))
    mid = slice(c.cu_l[1], c.cu_l[2])
    assert not o[mid].any() and torch.all(lse[mid] == -math.inf)
    s = D ** -0.5
    ref, p = c.reference(s), p_rounding(c, s, o.dtype)
    for b in (0, 2):
        sl = slice(c.cu_l[b], c.cu_l[b + 1])
        tol = ref[1][sl] + p[sl] + ref[0][sl].abs() * half_step(o.dtype) + 2.0 ** -24
        assert torch.all((o[sl].double().cpu() - ref[0][sl]).abs() <= tol)
        assert torch.all((lse[sl].double().cpu() - ref[2][sl]).abs() <= ref[3][sl])


@every_form
def test_scales(what, T, G, D, dt):
    for scale in (-0.3, 0.0, 1.5):
        c = Win([60, 0], [T, T], 33, 2, 2, G, D, 16, dt, seed=T, qscale=1.0)
        o, lse = run(c, scale=scale)
        check_tree(c, o, lse, c.reference(scale), p_rounding(c, scale, dt))


@every_form
@both_outputs
@pytest.mark.parametrize("how", ["grow", "leap", "fall"])
def test_scores_that_grow_and_fall_along_the_keys(what, T, G, D, dt, out, how):
    c = Win([900], [T], ALL, 0, 2, G, D, 64, dt, seed=T)
    for j in range(900 + T):
        f = {"grow": 2.0 ** (j // 100 - 4), "leap": 24.0 if j == 500 else 0.25, "fall": 2.0 ** (3 - j // 100)}[how]
        c.k[c.table_l[0][j // 64], :, j % 64] *= f
    o, lse = run(c, o_dtype=odt(dt, out))
    s = D ** -0.5
    check_tree(c, o, lse, c.reference(s), p_rounding(c, s, o.dtype))


@every_form
@both_outputs
@pytest.mark.parametrize("ctx", [300, 5000])
def test_keys_that_are_not_finite(what, T, G, D, dt, out, ctx):
    """A NaN key spoils the rows that see it and no others."""
    c = Win([ctx], [T], 64 if ctx == 300 else 4000, 2, 1, G, D, 16, dt, seed=D)
    o, lse = run(c, o_dtype=odt(dt, out))
    j = ctx + T // 2
    c.k[c.table_l[0][j // 16], :, j % 16, D - 3] = math.nan
    p, y = run(c, o_dtype=odt(dt, out))
    see = c.seen(0)[:, j].cuda()
    assert torch.equal(p[~see], o[~see]) and torch.equal(y[~see], lse[~see])
    assert torch.isnan(p[see]).all() and torch.isnan(y[see]).all()


@every_form
@both_outputs
def test_missing_pages(what, T, G, D, dt, out):
    """Pages that are needed and missing are left out and told, at a window's edge, inside and at the end."""
    c = Win([500, 40], [T, T], 300, 3, 1, G, D, 16, dt, seed=T)
    holes = [(500 - 290) // 16, 400 // 16, (500 + T - 1) // 16]
    for x, h in enumerate(holes):
        c.table[0, h] = c.k.shape[0] + 5 if x else -1
    c.dev()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = q.attn_window(c.cache, c.q.cuda(), c.table.cuda(), c.ctx, c.cu, T, window=300, sinks=3, status=st,
                           o_dtype=odt(dt, out))
    torch.cuda.synchronize()
    assert int(st) == 1
    see, rows = c.seen, c.rows
    gone = lambda n: torch.from_numpy(np.isin(np.arange(n) // 16, holes))  # noqa: E731
    c.seen = lambda b: see(b) & ~(gone(see(b).shape[1]) if b == 0 else torch.zeros(1, dtype=torch.bool))
    c.rows = lambda pool, b, h: torch.where(torch.isfinite(rows(pool, b, h)), rows(pool, b, h), 0.0)
    s = D ** -0.5
    check_tree(c, o, lse, c.reference(s), p_rounding(c, s, o.dtype))


@every_form
@both_outputs
def test_same_bits_and_odd_addresses(what, T, G, D, dt, out):
    """Outputs on a 16-byte boundary that is no 32-byte one, what lies around them, and repeats."""
    c = Win([2000, 11], [T, T - T // 3], 1500, 4, 2, G, D, 16, dt, seed=D)
    o, lse = run(c, o_dtype=odt(dt, out))
    n = o.numel()
    flat = torch.full((n + 64,), 7.0, dtype=o.dtype, device="cuda")
    at = 16 // flat.element_size()
    odd = flat[at:at + n].view(o.shape)
    assert odd.data_ptr() % 32 == 16
    for _ in range(3):
        odd.fill_(3.0)
        _, y = run(c, o=odd)
        assert torch.equal(odd, o) and torch.equal(y, lse) and torch.all(flat[:at] == 7) and torch.all(flat[at + n:] == 7)


@pytest.mark.parametrize("D,dt", [(64, BF), (128, FP)])
def test_a_long_prompt_among_more_than_32_sequences(D, dt):
    """The plan of one warp's sequences does not hold them: a thread counts each."""
    new = [1 + b % 3 for b in range(40)]
    new[17] = 3001
    ctx = [(b * 37) % 500 for b in range(40)]
    c = Win(ctx, new, 200, 4, 1, 4, D, 64, dt, seed=D)
    o, lse = run(c)
    s = D ** -0.5
    check_tree(c, o, lse, c.reference(s), p_rounding(c, s, dt))
