"""Outputs that share bytes with what other blocks still read, or with one another, are refused on
the host: whole arrays, slices that begin inside, and single elements at either end."""
import ctypes

import pytest

import int4_group_quantized_gs64_gb300 as q

EINVAL = -1
PAGES, PAGE, B, F, MP, N = 40, 16, 6, 5, 8, 23
# addresses far apart (aligned and never dereferenced: validation fails first)
AT = {n: 0x100000 * (i + 1) for i, n in enumerate(
    ("refs", "table", "lens", "more", "parent", "new_table", "new_lens", "moves", "ctx", "cu", "keep", "kept", "new_ctx"))}
BYTES = dict(refs=4 * PAGES, table=4 * B * MP, lens=4 * B, more=4 * B, parent=4 * F, new_table=4 * F * MP, new_lens=4 * F,
             moves=12 * F, ctx=4 * B, cu=4 * (B + 1), keep=4 * N, kept=4 * B, new_ctx=4 * B)
WS = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module")
def L():
    q.build()
    return q.lib()


def update(L, p):
    return L.attn_pages_update(p["refs"], PAGES, PAGE, p["table"], MP, p["lens"], p["more"], B, 9, 0, None, WS, 1 << 40,
                               None)


def fork(L, p):
    return L.attn_pages_fork(p["refs"], PAGES, PAGE, p["table"], MP, p["lens"], B, p["parent"], F, p["new_table"],
                             p["new_lens"], p["moves"], None, WS, 1 << 40, None)


def compact(L, p):
    d = q.AttnCacheDesc(0x10000, 0x10000, PAGES, 2, PAGE, 64, 1)
    return L.attn_compact(ctypes.byref(d), p["table"], MP, p["ctx"], p["cu"], B, N, p["keep"], p["kept"], None,
                          p["new_ctx"], None, None)


FORKED = ("new_table", "new_lens", "moves")
PAIRS = [(update, "table", x) for x in ("refs", "lens", "more")] + [(update, "refs", x) for x in ("lens", "more")]
PAIRS += [(fork, o, x) for o in FORKED for x in ("refs", "table", "lens", "parent")]
PAIRS += [(fork, "new_table", "new_lens"), (fork, "new_table", "moves"), (fork, "new_lens", "moves")]
PAIRS += [(compact, "new_ctx", x) for x in ("table", "ctx", "cu", "keep", "kept")]


@pytest.mark.parametrize("call,out,other", PAIRS, ids=[f"{c.__name__}-{o}-{x}" for c, o, x in PAIRS])
def test_shared_bytes_are_refused(L, call, out, other):
    for at in (0, BYTES[other] - 4, 4 - BYTES[out]):     # the same start; its last element; its first one
        p = {k: ctypes.c_void_p(v) for k, v in AT.items()}
        p[out] = ctypes.c_void_p(AT[other] + at)
        assert call(L, p) == EINVAL, at
