"""examples/stream_layer.py: prompts in chunks, drafts, forks and a window, against plain 64-bit
lists of each sequence's tokens."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
q = pytest.importorskip("int4_group_quantized_gs64_gb300")

from test_gpu_decode_layer import rotated  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "stream_layer.py")


def example():
    spec = importlib.util.spec_from_file_location("stream_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def normed(x, w):
    x = x.double()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()


def test_stream_against_lists(monkeypatch):
    """Attention outputs of every step against lists of normed, rotated keys and values that are
    kept, moved and copied as Python lists. Keys and queries are rounded to bf16 by both: where
    the last bits before it differ one may lie a step of 2^-8 off the other, so scores of
    magnitude up to s differ by 2^-7 s; the weights' own rounding and the output's are below."""
    ex = example()
    q.build()
    layer = ex.StreamAttention(B=3, H=256, Hq=6, Hkv=2, D=64, page=16, pages=64, max_len=640, window=70, sinks=5)
    D, Hkv, G, W, S = 64, 2, 3, layer.window, layer.sinks
    seen = {}
    window = q.attn_window

    def spy(*a, **k):
        seen["o"], seen["lse"] = window(*a, **k)
        return seen["o"], seen["lse"]
    monkeypatch.setattr(ex.qmv, "attn_window", spy)
    g = torch.Generator(device="cuda").manual_seed(5)
    rng = np.random.default_rng(5)
    empty = lambda: torch.zeros(0, Hkv, D, dtype=torch.float64, device="cuda")  # noqa: E731
    K, V = [empty() for _ in range(3)], [empty() for _ in range(3)]
    held = []

    def step(counts):
        n = sum(counts)
        h = torch.randn(n, 256, device="cuda", generator=g)
        layer.step(h, counts)
        o = seen["o"].view(n, Hkv, G, D).double()
        qkv = q.qmv_int4_gs(*layer.w_qkv, h).view(n, -1, D)
        at, new = 0, []
        for b, t in enumerate(counts):
            c = K[b].shape[0]
            p = torch.arange(c, c + t, device="cuda")
            x = qkv[at:at + t]
            qq = rotated(normed(x[:, :6], layer.q_norm), p, layer.inv_freq).to(torch.bfloat16).double().view(t, Hkv, G, D)
            kk = rotated(normed(x[:, 6:8], layer.k_norm), p, layer.inv_freq).to(torch.bfloat16).double()
            vv = x[:, 8:].to(torch.bfloat16).double()
            keys, vals = torch.cat([K[b], kk]), torch.cat([V[b], vv])
            j = torch.arange(c + t, device="cuda")
            back = p[:, None] - j
            see = (back >= 0) & ((back < W) | (j < S))
            s = torch.einsum("thgd,mhd->thgm", qq, keys) * D ** -0.5
            big = s.abs().max().item() if t else 0.0
            w = torch.softmax(s.masked_fill(~see[:, None, None], float("-inf")), -1)
            want = torch.einsum("thgm,mhd->thgd", w, vals)
            tol = (2.0 ** -7 * big + 2.0 ** -14) * torch.einsum("thgm,mhd->thgd", w, vals.abs())
            assert torch.all((o[at:at + t] - want).abs() <= tol), (b, t)
            new.append((keys, vals))
            at += t
        held.append(layer.held())
        return new

    for counts in ([100, 7, 33], [150, 0, 1], [5, 90, 17]):
        for b, (k, v) in enumerate(step(counts)):
            K[b], V[b] = k, v
        layer.accept_all()
    for i in range(24):
        B = len(K)
        counts = rng.integers(1, 7, B).tolist()
        new = step(counts)
        keep, kept = [], []
        for b, t in enumerate(counts):
            n = int(rng.integers(0 if i % 5 == 0 else 1, t + 1))
            path = np.sort(rng.choice(t, n, replace=False))
            keep += path.tolist() + [0] * (t - n)
            kept.append(n)
            at = torch.cat([torch.arange(len(K[b])), len(K[b]) + torch.from_numpy(path)]).to("cuda")
            K[b], V[b] = new[b][0][at], new[b][1][at]
        i32 = dict(dtype=torch.int32, device="cuda")
        layer.accept(torch.tensor(keep, **i32), torch.tensor(kept, **i32))
        assert layer.lens.tolist() == [len(k) for k in K]
        if i in (3, 10, 11, 18):
            parent = rng.integers(0, B, 4 if i < 12 else 2).tolist()
            layer.fork(parent)
            K, V = [K[p].clone() for p in parent], [V[p].clone() for p in parent]
    assert int(layer.status) == 0
    assert max(len(k) for k in K) > 2 * W
    # what a sequence can see, the pages at its edges, and what drafts may need
    assert max(held[3:]) <= 4 * ((W + S + 6) // 16 + 4)


def test_example_runs():
    out = subprocess.run([sys.executable, PATH, "--steps", "60"], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-2000:]
    assert "pages held" in out.stdout


@pytest.mark.parametrize("T", [1, 9])
def test_a_captured_step_takes_and_gives_back_pages(T):
    """Pages, append, attention and lengths of a step in one graph: replays follow the eager steps
    bit for bit while windows leave pages, others take them, and a page ends inside a step."""
    q.build()
    B, Hq, Hkv, D, page, W, S, pool = 5, 8, 2, 64, 16, 50, 3, 40
    N = B * T
    g = torch.Generator(device="cuda").manual_seed(T)
    inv = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    w = 1 + 0.1 * torch.randn(D, device="cuda", generator=g)
    cu = torch.arange(0, N + 1, T, dtype=torch.int32, device="cuda")
    more = torch.full((B,), T, dtype=torch.int32, device="cuda")

    class Side:
        def __init__(self):
            self.cache = q.AttnCache.empty(pool, Hkv, page, D, torch.bfloat16, "cuda")
            self.refs = torch.zeros(pool, dtype=torch.int32, device="cuda")
            self.table = torch.full((B, 64), -1, dtype=torch.int32, device="cuda")
            self.lens = torch.tensor([0, 3, 14, 15, 16], dtype=torch.int32, device="cuda")
            self.x = torch.zeros(N, Hq + 2 * Hkv, D, device="cuda")
            self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
            self.cache.k.zero_()
            self.cache.v.zero_()

        def step(self):
            q.attn_pages_update(self.refs, self.table, self.lens, more, page, window=W, sinks=S, status=self.st)
            a, k, v = self.x.split([Hq, Hkv, Hkv], 1)
            pos = (self.lens[:, None] + torch.arange(T, dtype=torch.int32, device="cuda")).view(-1)
            a = q.attn_norm_rope_append(self.cache, a, k, v, w, w, pos, inv, self.table, self.lens, cu, status=self.st)
            self.o, self.lse = q.attn_window(self.cache, a, self.table, self.lens, cu, T, window=W, sinks=S,
                                             status=self.st)
            self.lens += T

    one, two = Side(), Side()
    start = [t.clone() for t in (two.refs, two.table, two.lens)]
    two.step()          # (warm-up)
    for t, v in zip((two.refs, two.table, two.lens), start):
        t.copy_(v)
    two.cache.k.zero_(), two.cache.v.zero_(), two.st.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        two.step()
    for i in range(40):
        x = torch.randn(N, Hq + 2 * Hkv, D, device="cuda", generator=g)
        one.x.copy_(x), two.x.copy_(x)
        one.step()
        graph.replay()
        assert torch.equal(one.o, two.o) and torch.equal(one.lse, two.lse), i
        assert torch.equal(one.table, two.table) and torch.equal(one.refs, two.refs), i
        assert int(one.st) == int(two.st) == 0
    most = -(-(W + S + T) // page) + 3
    assert 0 < int(one.refs.sum()) <= B * most and int(one.refs.max()) == 1
