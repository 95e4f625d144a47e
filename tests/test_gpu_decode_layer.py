"""examples/decode_layer.py: drafting, accepting and evicting against a plain 64-bit form that
keeps every sequence's tokens as a list."""
import importlib.util
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
q = pytest.importorskip("int4_group_quantized_gs64_gb300")

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "decode_layer.py")


def example():
    spec = importlib.util.spec_from_file_location("decode_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rotated(x, pos, inv_freq):
    """Halves (i, i + D/2) of [n][heads][D] turned by pos * inv_freq, in 64 bits."""
    ang = pos.double()[:, None] * inv_freq
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = x.double().chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def test_layer_against_lists():
    """The cache of each sequence is mirrored as lists of rotated keys, values and sums.
    Keys and queries are rounded to bf16 by both (2^-9 each of a score's products at
    most, up to their own rounding's borders: a border's other side is a step of 2^-8,
    so scores of magnitude up to s differ by 2^-7 s where one crosses)."""
    ex = example()
    q.build()
    layer = ex.DecodeLayer(B=3, H=512, Hq=8, Hkv=2, D=64, E=16, I=128, limit=48, budget=24)
    B, T, D, Hkv, G = layer.B, layer.T, layer.D, layer.Hkv, layer.Hq // layer.Hkv
    g = torch.Generator(device="cuda").manual_seed(3)
    # per sequence and head: kept keys, values, sums
    K = [[torch.zeros(0, D, device="cuda", dtype=torch.float64) for _ in range(Hkv)] for _ in range(B)]
    V = [[t.clone() for t in row] for row in K]
    A = [[torch.zeros(0, device="cuda", dtype=torch.float64) for _ in range(Hkv)] for _ in range(B)]
    pos = [0] * B
    sees = torch.tensor([[bool(w >> d & 1) for d in range(T)] for w in ex.tree_mask()], device="cuda")
    evictions = 0
    for step in range(40):
        h = torch.randn(layer.N, 512, device="cuda", generator=g)
        h = h * torch.rsqrt(h.square().mean(-1, keepdim=True))
        o = layer.attention(h).view(B, T, Hkv, G, D).double()
        qkv = q.qmv_int4_gs(*layer.w_qkv, h).view(B, T, -1, D)
        n = torch.randint(1, 4, (B,), generator=g, device="cuda", dtype=torch.int32)
        for b in range(B):
            p = torch.tensor([pos[b] + d for d in ex.DEPTH], device="cuda")
            qq, kk, vv = qkv[b].split([layer.Hq, Hkv, Hkv], 1)
            qq = rotated(qq, p, layer.inv_freq).to(torch.bfloat16).double().view(T, Hkv, G, D)
            kk = rotated(kk, p, layer.inv_freq).to(torch.bfloat16).double()
            vv = vv.to(torch.bfloat16).double()
            for hd in range(Hkv):
                keys, vals = torch.cat([K[b][hd], kk[:, hd]]), torch.cat([V[b][hd], vv[:, hd]])
                x = torch.einsum("tgd,md->tgm", qq[:, hd], keys) * D ** -0.5
                c = len(K[b][hd])
                x[..., c:].masked_fill_(~sees[:, None], float("-inf"))
                w = torch.softmax(x, -1)
                want = torch.einsum("tgm,md->tgd", w, vals)
                big = x[x.isfinite()].abs().max().item()
                tol = (2.0 ** -7 * big + 2.0 ** -14) * torch.einsum("tgm,md->tgd", w, vals.abs())
                assert torch.all((o[b, :, hd] - want).abs() <= tol), (step, b, hd)
                sums = torch.cat([A[b][hd], torch.zeros(T, device="cuda", dtype=torch.float64)]) + w.sum((0, 1))
                m = c + int(n[b])
                K[b][hd], V[b][hd], A[b][hd] = keys[:m], vals[:m], sums[:m]
            pos[b] += int(n[b])
        old = layer.now
        lens = layer.ctx + n
        slots = layer.tables[old].long()
        sums = layer.sums[old][slots].transpose(1, 2).reshape(B, Hkv, -1)  # the sums as the layer has them
        if layer.accept(n):
            evictions += 1
            for b in range(B):
                m = int(lens[b])
                for hd in range(Hkv):
                    acc = sums[b, hd, :m]
                    assert torch.allclose(acc.double(), A[b][hd], rtol=2.0 ** -4, atol=2.0 ** -6)
                    if m > layer.budget:
                        mid = torch.argsort(acc[4:m - 16], descending=True, stable=True)[:layer.budget - 20] + 4
                        keep = torch.cat([torch.arange(4, device="cuda"), mid.sort().values,
                                          torch.arange(m - 16, m, device="cuda")])
                    else:
                        keep = torch.arange(m, device="cuda")
                    K[b][hd], V[b][hd], A[b][hd] = K[b][hd][keep], V[b][hd][keep], A[b][hd][keep]
        assert layer.ctx.tolist() == [len(K[b][0]) for b in range(B)] and layer.pos.tolist() == pos
    assert evictions >= 2 and int(layer.status) == 0


def test_example_runs():
    out = subprocess.run([sys.executable, PATH, "--steps", "40"], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-2000:]
    assert "evictions" in out.stdout
