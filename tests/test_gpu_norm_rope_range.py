"""Normed rotary append of heads whose squares leave fp32's range, and of sequences that do not fit,
on the GPU. The 64-bit form and its bound are those of test_gpu_norm_rope: a head that is scaled by a
power of two first has the same roundings, and what that takes from its smallest elements is below
D * 2^-149 of its largest."""
import math

import pytest

torch = pytest.importorskip("torch")
q = pytest.importorskip("int4_group_quantized_gs64_gb300")

from test_gpu_attn import BF, F32, Case  # noqa: E402
from test_gpu_norm_rope import call, check, inputs  # noqa: E402

pytestmark = pytest.mark.gpu
SCALES = (1e-45, 1e-42, 1e-39, 1e-37, 1e-30, 1e-23, 1e-22, 1e-20, 1e-17, 1e-12, 0.0, 1.0, 1e15, 3e18, 1e19, 1e25, 1e37)


@pytest.fixture(scope="module", autouse=True)
def _built():
    q.build()
    q.lib()


@pytest.mark.parametrize("Hkv,G,D,rot", [(2, 2, 64, 64), (2, 2, 64, 6), (4, 12, 64, 32), (1, 2, 128, 128),
                                         (2, 14, 128, 128), (2, 14, 128, 50)])
@pytest.mark.parametrize("src", [F32, BF])
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-30, 1e-6, 1e30])
def test_heads_of_any_magnitude(Hkv, G, D, rot, src, eps):
    """Few and many heads, the vector path and the other; neighbouring heads differ in magnitude."""
    eps = float(torch.tensor(eps, dtype=F32))
    c = Case([10], [len(SCALES)], Hkv, G, D, 16, BF, seed=D).dev()
    qkv, w, pos, inv = inputs(c, src, F32, rot)
    for n, s in enumerate(SCALES):
        for h in range(qkv.shape[1]):
            x = SCALES[(n + h) % len(SCALES)] if h % 3 else s
            qkv[n, h] = (qkv[n, h].double() * x).to(src)
    # values are copied, whatever they are: within the cache's range
    qkv[:, c.Hq + c.Hkv:] = 1.5
    out = call(c, qkv, w, pos, inv, eps=eps)
    torch.cuda.synchronize()
    check(c, out, qkv, w, pos, inv, rot, False, 1.0, eps)


@pytest.mark.parametrize("rot", [64, 6])
def test_values_keep_their_magnitude(rot):
    c = Case([3], [5], 2, 2, 64, 16, BF, seed=2).dev()
    qkv, w, pos, inv = inputs(c, F32, F32, rot)
    qkv[:, c.Hq + c.Hkv:] *= torch.tensor([1e-30, 1e-22, 1.0, 1e19, 1e30])[:, None, None]
    out = call(c, qkv, w, pos, inv, eps=0.0)
    torch.cuda.synchronize()
    check(c, out, qkv, w, pos, inv, rot, False, 1.0, 0.0)


@pytest.mark.parametrize("rot", [64, 6])
def test_one_large_element_and_many_small_ones(rot):
    """The small ones' squares are nothing beside it, they themselves are kept."""
    c = Case([3], [6], 2, 2, 64, 16, BF, seed=2).dev()
    qkv, w, pos, inv = inputs(c, F32, F32, rot)
    qkv[:3, :, 5] = 1e22
    qkv[:3] *= torch.tensor([1.0, 1e10, 1e-40])[:, None, None]
    qkv[3:] *= 1e-36
    qkv[3:, :, 7] *= torch.tensor([1e8, 1e14, 1.0])[:, None]
    qkv[:, c.Hq + c.Hkv:] = 0.25
    for eps in (0.0, 1e-6):
        out = call(c, qkv, w, pos, inv, eps=eps)
        torch.cuda.synchronize()
        check(c, out, qkv, w, pos, inv, rot, False, 1.0, eps)


@pytest.mark.parametrize("rot", [64, 6])
def test_infinities_and_nans_stay_in_their_head(rot):
    """inf / inf is NaN and x / inf zero; a NaN spoils its head."""
    c = Case([3], [4], 2, 2, 64, 16, BF, seed=2).dev()
    qkv, w, pos, inv = inputs(c, F32, None, rot)
    clean = call(c, qkv, w, pos, inv, eps=0.0).cpu()
    qkv[1, 2, 63], qkv[2, 0, 62] = math.inf, math.nan
    out = call(c, qkv, w, pos, inv, eps=0.0).cpu()
    same = torch.ones(4, c.Hq, dtype=torch.bool)
    same[1, 2] = same[2, 0] = False
    assert torch.equal(out[same], clean[same])
    assert torch.isnan(out[2, 0]).all()
    bad = torch.isnan(out[1, 2])
    assert bad[63] and not out[1, 2][~bad].any() and int(bad.sum()) == (2 if rot == 64 else 1)


@pytest.mark.parametrize("rot", [64, 6])
def test_sequences_that_do_not_fit(rot):
    """Status 2; their slots stay as they are, the other sequence's tokens arrive."""
    c = Case([20, 8, 5], [4, 4, 3], 1, 2, 64, 16, BF, seed=0).dev()
    qkv, w, pos, inv = inputs(c, BF, BF, rot)
    c.ctx.copy_(torch.tensor([20, c.width * 16 - 2, -1], dtype=torch.int32))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(c, qkv, w, pos, inv, status=st)
    torch.cuda.synchronize()
    changed = (c.cache.k.cpu() != c.k).flatten(1).any(1).nonzero().flatten().tolist()
    assert int(st) == 2 and changed == [c.table_l[0][1]]
    changed = (c.cache.v.cpu() != c.v).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [c.table_l[0][1]]
