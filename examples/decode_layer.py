"""One decoder layer that verifies drafted tokens, over a paged cache that it keeps short.

Every step takes a small tree of drafted tokens for each sequence through the
layer: the projections (int4 GEMVs), rotary positions and the append to the
cache, attention of the trees with the running attention weight of every cached
token, the output projection, and the routed experts. Some of the drafts are
accepted; where the cache would then outgrow its limit, the tokens that were
attended to least are evicted into the other of two page pools.

    python examples/decode_layer.py            # prints what the cache held, and us a step

Weights and hidden states are seeded random numbers; norms, residuals and the
acceptance are plain torch.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

import datagen
import int4_group_quantized_gs64_gb300 as qmv

# A tree of four drafts, the likeliest path first, so that what is accepted of it
# lies at the front of the drafts' slots:
#     0 - 1 - 2
#      \- 3
PARENT = [-1, 0, 1, 0]
DEPTH = [0, 1, 2, 1]


def tree_mask():
    """A word a draft: bit d set where d is the draft itself or one of its ancestors."""
    words = []
    for t, p in enumerate(PARENT):
        words.append((words[p] if p >= 0 else 0) | 1 << t)
    return words


class DecodeLayer:
    def __init__(self, B=4, H=1024, Hq=16, Hkv=4, D=64, E=32, I=256, top_k=4, page=16, limit=96,
                 budget=64, dtype=torch.bfloat16, device="cuda"):
        self.B, self.Hq, self.Hkv, self.D, self.top_k = B, Hq, Hkv, D, top_k
        self.limit, self.budget, self.T = limit, budget, len(PARENT)
        self.N = B * self.T

        def matrix(rows, cols, seed):  # int4 rows of about unit gain
            wq, sc, _ = datagen.dense_int4(rows, cols, 1, seed=seed)
            return torch.from_numpy(wq).to(device), torch.from_numpy(sc * (10 / cols ** 0.5)).to(device)

        self.w_qkv = matrix((Hq + 2 * Hkv) * D, H, 11)
        self.w_out = matrix(H, Hq * D, 12)
        moe = datagen.moe_weights(E, H, I, seed=13)
        self.moe = qmv.MoeInt4Weights.from_numpy(moe, device)
        self.w_router = torch.from_numpy(datagen.normal_f32(21, (H, E), std=H ** -0.5, seed=14)).to(device)
        self.inv_freq = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).to(device)

        # two pools of pages: the layer reads one, and evicts into the other
        pages_each = -(-(limit + self.T) // page)
        i32 = dict(dtype=torch.int32, device=device)
        self.pools = [qmv.AttnCache.empty(B * pages_each, Hkv, page, D, dtype, device) for _ in range(2)]
        self.sums = [torch.zeros(B * pages_each, Hkv, page, device=device) for _ in range(2)]
        order = torch.from_numpy(np.random.default_rng(15).permutation(B * pages_each)).to(**i32)
        self.tables = [order.view(B, pages_each), order.flip(0).view(B, pages_each)]
        self.now = 0
        self.ctx = torch.zeros(B, **i32)  # cached tokens
        self.pos = torch.zeros(B, **i32)  # tokens so far: a position outlives its neighbours
        self.held = 0                     # an upper bound of ctx that the host keeps

        self.cu = torch.arange(0, self.N + 1, self.T, **i32)
        self.mask = torch.tensor(tree_mask() * B, **i32).view(self.N, 1)
        self.depth = torch.tensor(DEPTH * B, **i32)
        self.status = torch.zeros(1, **i32)
        self.ws = torch.empty(max(256, qmv.attn_tree_workspace_bytes(
            self.pools[0], Hq, B, self.N, self.T, pages_each, True)), dtype=torch.uint8, device=device)

    def attention(self, h):
        """Attention of the drafted tokens' normed states h [N][H]; appends them to the cache."""
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        cache, table, sums = self.pools[self.now], self.tables[self.now], self.sums[self.now]
        qkv = qmv.qmv_int4_gs(*self.w_qkv, h)
        q, k, v = qkv.view(self.N, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], 1)
        pos = self.pos.repeat_interleave(self.T, output_size=self.N) + self.depth
        q = qmv.attn_rope_append(cache, q, k, v, pos, self.inv_freq, table, self.ctx, self.cu,
                                 acc=sums, status=self.status)
        o, _ = qmv.attn_tree(cache, q, table, self.ctx, self.cu, self.T, mask=self.mask,
                             o_dtype=torch.float32, acc=sums, ws=self.ws, status=self.status)
        return o

    def step(self, x):
        """The layer's output for the drafted tokens' states x [N][H]."""
        norm = lambda t: t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)
        o = self.attention(norm(x))
        x = x + qmv.qmv_int4_gs(*self.w_out, o.view(self.N, -1))
        h = norm(x)
        out, _, _ = qmv.moe_route_expert_ffn_int4(self.moe, h @ self.w_router, h, self.top_k)
        return x + norm(out)

    def accept(self, n):
        """Keeps the first n[b] drafts of each sequence (int32 [B], 1 .. 3), and evicts when the
        cache would outgrow its limit."""
        self.ctx = self.ctx + n
        self.pos = self.pos + n
        self.held += 3
        if self.held > self.limit - self.T:
            old, new = self.now, 1 - self.now
            _, self.ctx = qmv.attn_evict(self.pools[old], self.sums[old], self.tables[old], self.ctx,
                                         self.budget, self.pools[new], self.sums[new],
                                         self.tables[new], sink=4, recent=16, status=self.status)
            self.now, self.held = new, self.budget
            return True
        return False


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    layer = DecodeLayer()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(layer.N, layer.moe.H, device="cuda", generator=g)
    evicted, start, end = 0, torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(a.steps + 10):
        if i == 10:
            start.record()
        y = layer.step(x)
        evicted += layer.accept(torch.randint(1, 4, (layer.B,), device="cuda", generator=g, dtype=torch.int32))
        x = y + 0.5 * torch.randn(y.shape, device="cuda", generator=g)
    end.record()
    torch.cuda.synchronize()
    if int(layer.status):
        raise SystemExit(f"device status {int(layer.status)}")
    print(f"{a.steps + 10} steps of {layer.B} trees of {layer.T} drafts: positions {layer.pos.tolist()}, "
          f"cached {layer.ctx.tolist()}, {evicted} evictions, {start.elapsed_time(end) / a.steps * 1e3:.0f} us a step")


if __name__ == "__main__":
    main()
