"""Streaming attention of one layer: prompts in chunks, forks, drafts, and a bounded cache.

Every sequence sees the last WINDOW tokens and its first SINKS ones, so its pages in between
are given back as it grows and the pool stays small. A step takes new tokens (a chunk of a
prompt, or a chain of drafts) through the attention of a layer: pages for them, the norms of
queries and keys with rotary positions and the append, attention over the window, and, after
drafts, the accepted ones moved to the front. fork() continues a sequence in several ways: the
children share its whole pages.

    python examples/stream_layer.py            # prints what the sequences held, and us a step

Weights and hidden states are seeded random numbers; which drafts are accepted is random too.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import datagen
import int4_group_quantized_gs64_gb300 as qmv


class StreamAttention:
    def __init__(self, B=4, H=512, Hq=8, Hkv=2, D=64, page=16, pages=256, max_len=4096, window=200, sinks=4,
                 dtype=torch.bfloat16, device="cuda"):
        self.H, self.Hq, self.Hkv, self.D, self.page = H, Hq, Hkv, D, page
        self.window, self.sinks, self.dtype, self.device = window, sinks, dtype, device

        def matrix(rows, cols, seed):  # int4 rows of about unit gain
            wq, sc, _ = datagen.dense_int4(rows, cols, 1, seed=seed)
            return torch.from_numpy(wq).to(device), torch.from_numpy(sc * (10 / cols ** 0.5)).to(device)

        self.w_qkv = matrix((Hq + 2 * Hkv) * D, H, 21)
        self.w_out = matrix(H, Hq * D, 22)
        g = torch.Generator(device=device).manual_seed(23)
        self.q_norm, self.k_norm = (1 + 0.2 * torch.randn(D, device=device, generator=g) for _ in range(2))
        self.inv_freq = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).to(device)
        self.cache = qmv.AttnCache.empty(pages, Hkv, page, D, dtype, device)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=device)
        self.table = torch.full((B, -(-max_len // page)), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(B, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def step(self, h, counts):
        """Attention of new tokens' normed states h [N][H], counts[b] of them a sequence (a list);
        returns the output projection's [N][H]. The tokens are in the cache, not yet in lens."""
        N, B, T = h.shape[0], len(counts), max(counts)
        more = torch.tensor(counts, dtype=torch.int32, device=self.device)
        cu = torch.zeros(B + 1, dtype=torch.int32, device=self.device)
        cu[1:] = more.cumsum(0)
        qmv.attn_pages_update(self.refs, self.table, self.lens, more, self.page, window=self.window,
                              sinks=self.sinks, status=self.status)
        qkv = qmv.qmv_int4_gs(*self.w_qkv, h)
        q, k, v = qkv.view(N, -1, self.D).split([self.Hq, self.Hkv, self.Hkv], 1)
        first = (self.lens - cu[:-1]).repeat_interleave(more.long(), output_size=N)
        pos = first + torch.arange(N, dtype=torch.int32, device=self.device)
        q = qmv.attn_norm_rope_append(self.cache, q, k, v, self.q_norm, self.k_norm, pos, self.inv_freq,
                                      self.table, self.lens, cu, status=self.status)
        o, _ = qmv.attn_window(self.cache, q, self.table, self.lens, cu, T, window=self.window,
                               sinks=self.sinks, o_dtype=torch.float32, status=self.status)
        self.cu = cu
        return qmv.qmv_int4_gs(*self.w_out, o.view(N, -1))

    def accept_all(self):
        self.lens = self.lens + (self.cu[1:] - self.cu[:-1])

    def accept(self, keep, kept):
        """Keeps, of each sequence's last new tokens, those at keep (int32 [N], kept[b] of them from
        cu[b] on, ascending)."""
        self.lens = qmv.attn_compact(self.cache, self.table, self.lens, self.cu, keep, kept, status=self.status)

    def fork(self, parent):
        """Goes on with children of the sequences (a list of rows) in their place."""
        parent = torch.tensor(parent, dtype=torch.int32, device=self.device)
        table, lens, moves = qmv.attn_pages_fork(self.refs, self.table, self.lens, parent, self.page,
                                                 status=self.status)
        qmv.attn_pages_copy(self.cache, self.cache, moves, status=self.status)
        gone = torch.zeros_like(self.lens)       # the parents' own hold ends
        qmv.attn_pages_update(self.refs, self.table, gone, gone, self.page, status=self.status)
        self.table, self.lens = table, lens

    def held(self):
        return int((self.refs > 0).sum())


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    layer = StreamAttention()
    g = torch.Generator(device="cuda").manual_seed(1)
    states = lambda n: torch.randn(n, layer.H, device="cuda", generator=g)  # noqa: E731
    for chunk in ([300, 120, 33, 7], [300, 0, 250, 1]):          # prompts
        layer.step(states(sum(chunk)), chunk)
        layer.accept_all()
    most, T = layer.held(), 4
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(a.steps):
        if i == min(10, a.steps - 1):
            start.record()
        B = layer.lens.shape[0]
        layer.step(states(B * T), [T] * B)                       # chains of drafts
        kept = torch.randint(1, T + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
        keep = torch.rand(B, T, device="cuda", generator=g).argsort(1).argsort(1) < kept[:, None]
        layer.accept(torch.where(keep, torch.arange(T, device="cuda"), T).sort(1).values.int().view(-1), kept)
        if i % 25 == 24:
            layer.fork([0, 0, 1, 2])
        if i % 10 == 0:
            most = max(most, layer.held())
    end.record()
    torch.cuda.synchronize()
    if int(layer.status):
        raise SystemExit(f"device status {int(layer.status)}")
    n = max(1, a.steps - 10)
    print(f"{a.steps} steps: lengths {layer.lens.tolist()}, {layer.held()} pages held, {most} at most, "
          f"{start.elapsed_time(end) / n * 1e3:.0f} us a step")


if __name__ == "__main__":
    main()
