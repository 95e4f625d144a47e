"""The attention entry points refuse bad arguments on the host, before any CUDA call."""
import ctypes

import pytest

import int4_group_quantized_gs64_gb300 as q

EINVAL, ESHAPE, EWORKSPACE, EALIGN = -1, -2, -3, -6
FAKE = 0x10000  # aligned and never dereferenced: validation fails first
P = ctypes.c_void_p(FAKE)
ODD = ctypes.c_void_p(FAKE + 2)


@pytest.fixture(scope="module")
def L():
    q.build()
    return q.lib()


def desc(k=FAKE, v=FAKE, pages=8, Hkv=2, page=16, D=64, dtype=1):
    return q.AttnCacheDesc(k, v, pages, Hkv, page, D, dtype)


def rope(L, d=None, **kw):
    a = dict(q=P, qs=256, k=P, ks=128, v=P, vs=128, t=1, Hq=4, pos=P, f=P, rot=64, inter=0, m=1.0,
             table=P, mp=4, ctx=P, cu=P, B=2, N=3, out=P, acc=None, st=None)
    a.update(kw)
    return L.attn_rope_append(ctypes.byref(d or desc()), a["q"], a["qs"], a["k"], a["ks"], a["v"],
                              a["vs"], a["t"], a["Hq"], a["pos"], a["f"], a["rot"], a["inter"],
                              a["m"], a["table"], a["mp"], a["ctx"], a["cu"], a["B"], a["N"],
                              a["out"], a["acc"], a["st"], None)


def tree(L, d=None, **kw):
    a = dict(q=P, qs=256, Hq=4, table=P, mp=4, ctx=P, cu=P, B=2, N=3, T=2, mask=P, words=1, scale=0.1,
             o=P, ot=1, lse=P, ai=None, ao=None, decay=1.0, st=None, ws=P, wb=1 << 40)
    a.update(kw)
    return L.attn_tree(ctypes.byref(d or desc()), a["q"], a["qs"], a["Hq"], a["table"], a["mp"],
                       a["ctx"], a["cu"], a["B"], a["N"], a["T"], a["mask"], a["words"], a["scale"],
                       a["o"], a["ot"], a["lse"], a["ai"], a["ao"], a["decay"], a["st"], a["ws"],
                       a["wb"], None)


def evict(L, d=None, e=None, **kw):
    a = dict(acc=P, table=P, mp=4, lens=P, B=2, budget=8, sink=1, recent=2, dacc=P,
             dt=ctypes.c_void_p(FAKE + 64), dmp=1, keep=P, nl=P, st=None)
    a.update(kw)
    return L.attn_evict(ctypes.byref(d or desc()), a["acc"], a["table"], a["mp"], a["lens"], a["B"],
                        a["budget"], a["sink"], a["recent"], ctypes.byref(e or desc()), a["dacc"],
                        a["dt"], a["dmp"], a["keep"], a["nl"], a["st"], None)


@pytest.mark.parametrize("call", [rope, tree, evict], ids=["rope", "tree", "evict"])
@pytest.mark.parametrize("bad,want", [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(pages=0), EINVAL), (dict(Hkv=0), EINVAL),
    (dict(dtype=0), EINVAL), (dict(dtype=3), EINVAL), (dict(D=96), ESHAPE), (dict(D=256), ESHAPE),
    (dict(page=8), ESHAPE), (dict(page=48), ESHAPE), (dict(page=512), ESHAPE),
    (dict(pages=1 << 26), ESHAPE), (dict(k=FAKE + 8), EALIGN), (dict(v=FAKE + 2), EALIGN)])
def test_cache_descriptor(L, call, bad, want):
    assert call(L, desc(**bad)) == want


@pytest.mark.parametrize("call", [rope, tree, evict], ids=["rope", "tree", "evict"])
def test_batch_limits(L, call):
    assert call(L, B=-1) == EINVAL
    assert call(L, mp=0) == EINVAL
    assert call(L, B=40000) == ESHAPE          # 40000 * 2 heads
    assert call(L, mp=(1 << 26) + 1) == ESHAPE  # * 16 > 2^30
    assert call(L, B=0) == 0                    # nothing to do


def test_rope(L):
    for k in ("q", "k", "v", "pos", "f", "table", "ctx", "cu", "out"):
        assert rope(L, **{k: None}) == EINVAL, k
    assert rope(L, N=-1) == EINVAL and rope(L, N=0) == 0 and rope(L, N=(1 << 22) + 1) == ESHAPE
    assert rope(L, Hq=3) == EINVAL and rope(L, Hq=0) == EINVAL and rope(L, Hq=2048) == EINVAL
    for r in (0, 1, 33, 66):
        assert rope(L, rot=r) == EINVAL, r
    assert rope(L, m=float("inf")) == EINVAL and rope(L, m=float("nan")) == EINVAL
    assert rope(L, t=2) == EINVAL and rope(L, t=7) == EINVAL     # fp16 into a bf16 cache
    assert rope(L, qs=255) == ESHAPE and rope(L, ks=127) == ESHAPE and rope(L, vs=0) == ESHAPE
    odd1 = ctypes.c_void_p(FAKE + 1)
    assert rope(L, q=odd1) == EALIGN and rope(L, t=0, k=ODD) == EALIGN
    assert rope(L, f=ctypes.c_void_p(FAKE + 4)) == EALIGN
    assert rope(L, out=ctypes.c_void_p(FAKE + 8)) == EALIGN
    for k in ("pos", "table", "ctx", "cu", "acc", "st"):
        assert rope(L, **{k: ODD}) == EALIGN, k


def test_tree(L):
    for k in ("q", "table", "ctx", "cu", "o", "lse"):
        assert tree(L, **{k: None}) == EINVAL, k
    assert tree(L, N=-1) == EINVAL and tree(L, N=0) == 0
    assert tree(L, Hq=3) == EINVAL and tree(L, T=0) == EINVAL and tree(L, T=257) == ESHAPE
    assert tree(L, words=0) == ESHAPE and tree(L, T=33) == ESHAPE and tree(L, words=9) == ESHAPE
    assert tree(L, scale=float("nan")) == EINVAL and tree(L, decay=float("inf")) == EINVAL
    assert tree(L, ot=2) == EINVAL and tree(L, ot=9) == EINVAL
    assert tree(L, qs=255) == ESHAPE and tree(L, qs=260) == EALIGN
    assert tree(L, ai=P) == EINVAL             # weights in, nowhere to put them
    for k in ("q", "o"):
        assert tree(L, **{k: ctypes.c_void_p(FAKE + 8)}) == EALIGN, k
    for k in ("table", "ctx", "cu", "mask", "lse", "ao", "st"):
        assert tree(L, **{k: ODD}) == EALIGN, k
    d = desc()
    need = L.attn_tree_workspace_bytes(ctypes.byref(d), 4, 2, 3, 2, 4, 0)
    assert need > 0 and need % 256 == 0
    assert tree(L, ws=None) == EWORKSPACE and tree(L, wb=need - 1) == EWORKSPACE
    assert tree(L, ws=ctypes.c_void_p(FAKE + 128)) == EWORKSPACE
    assert L.attn_tree_workspace_bytes(ctypes.byref(desc(D=96)), 4, 2, 3, 2, 4, 0) == 0
    assert L.attn_tree_workspace_bytes(ctypes.byref(d), 3, 2, 3, 2, 4, 0) == 0
    assert L.attn_tree_workspace_bytes(ctypes.byref(d), 4, 2, 3, 257, 4, 0) == 0


def test_evict(L):
    for k in ("acc", "table", "lens", "dacc", "dt", "keep", "nl"):
        assert evict(L, **{k: None}) == EINVAL, k
    assert evict(L, budget=0) == EINVAL and evict(L, sink=-1) == EINVAL
    assert evict(L, recent=-1) == EINVAL and evict(L, sink=5, recent=4) == EINVAL
    assert evict(L, e=desc(Hkv=1)) == ESHAPE and evict(L, e=desc(D=128)) == ESHAPE
    assert evict(L, e=desc(dtype=2)) == ESHAPE and evict(L, e=desc(page=24)) == ESHAPE
    assert evict(L, dmp=0) == EINVAL
    assert evict(L, dt=P) == EINVAL            # onto the source's own pages
    for k in ("acc", "table", "lens", "dacc", "dt", "keep", "nl", "st"):
        assert evict(L, **{k: ODD}) == EALIGN, k


def test_binding_checks():
    torch = pytest.importorskip("torch")
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        q.AttnCache(k, k)                      # not on the GPU
    with pytest.raises(TypeError):
        q.AttnCache(k.float(), k.float())
