"""Normed append, windowed attention and the upkeep of pages refuse bad arguments on the host,
before any CUDA call."""
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


def norm(L, d=None, **kw):
    a = dict(q=P, qs=256, k=P, ks=128, v=P, vs=128, t=1, Hq=4, qw=P, kw=P, wt=0, eps=1e-6, pos=P, f=P,
             rot=64, inter=0, m=1.0, table=P, mp=4, ctx=P, cu=P, B=2, N=3, out=P, acc=None, st=None)
    a.update(kw)
    return L.attn_norm_rope_append(ctypes.byref(d or desc()), a["q"], a["qs"], a["k"], a["ks"], a["v"],
                                   a["vs"], a["t"], a["Hq"], a["qw"], a["kw"], a["wt"], a["eps"],
                                   a["pos"], a["f"], a["rot"], a["inter"], a["m"], a["table"], a["mp"],
                                   a["ctx"], a["cu"], a["B"], a["N"], a["out"], a["acc"], a["st"], None)


def window(L, d=None, **kw):
    a = dict(q=P, qs=256, Hq=4, table=P, mp=4, ctx=P, cu=P, B=2, N=3, T=2, W=9, S=1, scale=0.1, o=P, ot=1,
             lse=P, st=None, ws=P, wb=1 << 40)
    a.update(kw)
    return L.attn_window(ctypes.byref(d or desc()), a["q"], a["qs"], a["Hq"], a["table"], a["mp"], a["ctx"],
                         a["cu"], a["B"], a["N"], a["T"], a["W"], a["S"], a["scale"], a["o"], a["ot"],
                         a["lse"], a["st"], a["ws"], a["wb"], None)


def compact(L, d=None, **kw):
    a = dict(table=P, mp=4, ctx=P, cu=P, B=2, N=3, keep=P, kept=P, acc=None, out=ctypes.c_void_p(FAKE + 64),
             st=None)
    a.update(kw)
    return L.attn_compact(ctypes.byref(d or desc()), a["table"], a["mp"], a["ctx"], a["cu"], a["B"], a["N"],
                          a["keep"], a["kept"], a["acc"], a["out"], a["st"], None)


CACHE_CALLS = {"norm": norm, "window": window, "compact": compact}


@pytest.mark.parametrize("call", CACHE_CALLS.values(), ids=CACHE_CALLS.keys())
@pytest.mark.parametrize("bad,want", [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(pages=0), EINVAL), (dict(Hkv=0), EINVAL),
    (dict(dtype=0), EINVAL), (dict(dtype=3), EINVAL), (dict(D=96), ESHAPE), (dict(D=256), ESHAPE),
    (dict(page=8), ESHAPE), (dict(page=48), ESHAPE), (dict(page=512), ESHAPE),
    (dict(pages=1 << 26), ESHAPE), (dict(k=FAKE + 8), EALIGN), (dict(v=FAKE + 2), EALIGN)])
def test_cache_descriptor(L, call, bad, want):
    assert call(L, desc(**bad)) == want


@pytest.mark.parametrize("call", CACHE_CALLS.values(), ids=CACHE_CALLS.keys())
def test_batch_limits(L, call):
    assert call(L, B=-1) == EINVAL
    assert call(L, mp=0) == EINVAL
    assert call(L, B=40000) == ESHAPE          # 40000 * 2 heads
    assert call(L, mp=(1 << 26) + 1) == ESHAPE  # * 16 > 2^30
    assert call(L, B=0) == 0                    # nothing to do


def test_norm(L):
    for k in ("q", "k", "v", "pos", "f", "table", "ctx", "cu", "out"):
        assert norm(L, **{k: None}) == EINVAL, k
    assert norm(L, N=0) == 0 and norm(L, N=-1) == EINVAL and norm(L, N=(1 << 22) + 1) == ESHAPE
    assert norm(L, wt=2) == EINVAL and norm(L, wt=5) == EINVAL    # fp16 weights of a bf16 cache
    for eps in (-1e-9, float("inf"), float("nan")):
        assert norm(L, eps=eps) == EINVAL
    assert norm(L, rot=33) == EINVAL and norm(L, t=2) == EINVAL and norm(L, Hq=3) == EINVAL
    assert norm(L, qs=255) == ESHAPE
    assert norm(L, qw=ODD) == EALIGN and norm(L, kw=ODD) == EALIGN
    odd1 = ctypes.c_void_p(FAKE + 1)
    assert norm(L, qw=odd1, wt=1) == EALIGN and norm(L, kw=odd1, wt=1) == EALIGN
    for k in ("pos", "table", "ctx", "cu", "acc", "st"):
        assert norm(L, **{k: ODD}) == EALIGN, k


def test_window(L):
    for k in ("q", "table", "ctx", "cu", "o", "lse"):
        assert window(L, **{k: None}) == EINVAL, k
    assert window(L, N=-1) == EINVAL and window(L, N=0) == 0 and window(L, N=(1 << 22) + 1) == ESHAPE
    assert window(L, Hq=3) == EINVAL and window(L, T=0) == EINVAL and window(L, T=(1 << 22) + 1) == ESHAPE
    assert window(L, T=1 << 22, Hq=1024, qs=1 << 20) == ESHAPE       # 2^22 * 512 rows
    assert window(L, W=0) == EINVAL and window(L, W=-5) == EINVAL and window(L, S=-1) == EINVAL
    assert window(L, scale=float("nan")) == EINVAL and window(L, scale=float("inf")) == EINVAL
    assert window(L, ot=2) == EINVAL and window(L, ot=9) == EINVAL
    assert window(L, qs=255) == ESHAPE and window(L, qs=260) == EALIGN
    for k in ("q", "o"):
        assert window(L, **{k: ctypes.c_void_p(FAKE + 8)}) == EALIGN, k
    for k in ("table", "ctx", "cu", "lse", "st"):
        assert window(L, **{k: ODD}) == EALIGN, k
    d = desc()
    for T in (2, 100, 1 << 20):
        need = L.attn_window_workspace_bytes(ctypes.byref(d), 4, 2, 3, T, 4)
        assert need > 0 and need % 256 == 0
        assert window(L, T=T, ws=None) == EWORKSPACE and window(L, T=T, wb=need - 1) == EWORKSPACE
        assert window(L, T=T, ws=ctypes.c_void_p(FAKE + 128)) == EWORKSPACE
    assert L.attn_window_workspace_bytes(ctypes.byref(desc(D=96)), 4, 2, 3, 2, 4) == 0
    assert L.attn_window_workspace_bytes(ctypes.byref(d), 3, 2, 3, 2, 4) == 0
    assert L.attn_window_workspace_bytes(ctypes.byref(d), 4, 2, 3, 0, 4) == 0


def test_compact(L):
    for k in ("table", "ctx", "cu", "keep", "kept", "out"):
        assert compact(L, **{k: None}) == EINVAL, k
    assert compact(L, N=-1) == EINVAL
    assert compact(L, out=P) == EINVAL             # onto ctx
    for k in ("table", "ctx", "cu", "keep", "kept", "acc", "out", "st"):
        assert compact(L, **{k: ODD}) == EALIGN, k


def update(L, **kw):
    a = dict(refs=P, pages=8, page=16, table=P, mp=4, lens=P, more=P, B=2, W=9, S=0, st=None, ws=P, wb=1 << 40)
    a.update(kw)
    return L.attn_pages_update(a["refs"], a["pages"], a["page"], a["table"], a["mp"], a["lens"], a["more"],
                               a["B"], a["W"], a["S"], a["st"], a["ws"], a["wb"], None)


def fork(L, **kw):
    a = dict(refs=P, pages=8, page=16, table=P, mp=4, lens=P, B=2, parent=P, F=3, nt=ctypes.c_void_p(FAKE + 64),
             nl=ctypes.c_void_p(FAKE + 64), moves=P, st=None, ws=P, wb=1 << 40)
    a.update(kw)
    return L.attn_pages_fork(a["refs"], a["pages"], a["page"], a["table"], a["mp"], a["lens"], a["B"],
                             a["parent"], a["F"], a["nt"], a["nl"], a["moves"], a["st"], a["ws"], a["wb"], None)


def copy(L, d=None, e=None, **kw):
    a = dict(moves=P, n=2, sa=None, da=None, st=None)
    a.update(kw)
    return L.attn_pages_copy(ctypes.byref(d or desc()), ctypes.byref(e or desc()), a["moves"], a["n"], a["sa"],
                             a["da"], a["st"], None)


@pytest.mark.parametrize("call,rows", [(update, "B"), (fork, "F"), (fork, "B")])
def test_pages_limits(L, call, rows):
    assert call(L, pages=0) == EINVAL and call(L, pages=(1 << 30) + 1) == ESHAPE
    assert call(L, mp=0) == EINVAL and call(L, mp=(1 << 26) + 1) == ESHAPE
    for page in (0, 8, 24, 512, -16):
        assert call(L, page=page) == ESHAPE
    assert call(L, **{rows: -1}) == EINVAL and call(L, **{rows: 65536}) == ESHAPE
    assert call(L, **{rows: 65535}, mp=32769) == ESHAPE             # 2^31 entries
    for k in ("refs", "table", "lens"):
        assert call(L, **{k: None}) == EINVAL, k
    for k in ("refs", "table", "lens", "st"):
        assert call(L, **{k: ODD}) == EALIGN, k


def test_pages_update(L):
    assert update(L, B=0) == 0 and update(L, more=None) == EINVAL and update(L, more=ODD) == EALIGN
    assert update(L, W=0) == EINVAL and update(L, S=-1) == EINVAL
    need = L.attn_pages_update_workspace_bytes(8, 2, 4)
    assert need > 0 and need % 256 == 0
    assert update(L, wb=need - 1) == EWORKSPACE and update(L, ws=None) == EWORKSPACE
    assert update(L, ws=ctypes.c_void_p(FAKE + 4)) == EWORKSPACE
    assert L.attn_pages_update_workspace_bytes(0, 2, 4) == 0


def test_pages_fork(L):
    assert fork(L, F=0) == 0
    for k in ("parent", "nt", "nl", "moves"):
        assert fork(L, **{k: None}) == EINVAL, k
        assert fork(L, **{k: ODD}) == EALIGN, k
    assert fork(L, nt=P) == EINVAL and fork(L, nl=P) == EINVAL      # onto the parents'
    need = L.attn_pages_fork_workspace_bytes(8, 3)
    assert need > 0 and need % 256 == 0
    assert fork(L, wb=need - 1) == EWORKSPACE and fork(L, ws=None) == EWORKSPACE


def test_pages_copy(L):
    assert copy(L, n=0) == 0 and copy(L, n=-1) == EINVAL and copy(L, moves=None) == EINVAL
    assert copy(L, n=1 << 30) == ESHAPE
    assert copy(L, sa=P) == EINVAL                                  # weights to nowhere
    for bad in (dict(Hkv=1), dict(D=128), dict(dtype=2), dict(page=32)):
        assert copy(L, None, desc(**bad)) == ESHAPE
    assert copy(L, desc(D=96)) == ESHAPE and copy(L, None, desc(k=None)) == EINVAL
    for k in ("moves", "da", "st"):
        assert copy(L, **{k: ODD}) == EALIGN, k
    assert copy(L, sa=ODD, da=P) == EALIGN


def test_outputs_onto_what_other_blocks_read(L):
    other = ctypes.c_void_p(FAKE + 128)
    assert fork(L, parent=other, nl=other) == EINVAL
    for k in ("ctx", "keep", "kept"):
        assert compact(L, **{k: other, "out": other}) == EINVAL, k
