"""An attention layer on NVFP4 weights and a 4-bit key and value cache.

Projects, rotates, writes the cache and attends: first a batch of prompts of different lengths, then
single tokens, each step in a CUDA graph.  The outputs are compared with the same layer in fp32, on
the values that the cache holds.

    python examples/attention_layer.py [steps]
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import nvfp4_block_scaled_gemv_gb300 as nv  # noqa: E402


class Layer:
    """Fused query, key and value projection, attention, output projection."""

    def __init__(self, hidden=1024, heads=16, kv_heads=4, head_dim=64, pages=64, page_size=32, max_pages=12, seed=0,
                 device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.head_dim, self.page_size = heads, kv_heads, head_dim, page_size
        self.encode_w, self.encode_x = 64.0, 1.0
        rows = (heads + 2 * kv_heads) * head_dim

        def weights(m, k):
            return nv.quantize(torch.randn((1, m, k), device=device, generator=g) / k ** 0.5, self.encode_w)

        self.w_in, self.s_in = weights(rows, hidden)
        self.w_out, self.s_out = weights(hidden, heads * head_dim)
        self.table = nv.rope_table(head_dim, base=10000.0, scaling="bands", factor=8.0, original=8192, low=1.0, high=4.0,
                                   device=device)
        # keys and values are brought to the middle of the scales' range
        self.encode_k = torch.full((kv_heads,), 4.0, device=device)
        self.encode_v = torch.full((kv_heads,), 8.0, device=device)
        self.cache = nv.kv_cache(pages, kv_heads, head_dim, page_size, device=device)
        self.max_pages = max_pages

    def project(self, x, weights, scales):
        q, s = nv.quantize(x, self.encode_x)
        return nv.gemm(weights, q.unsqueeze(0), scales, s, alpha=1 / (self.encode_w * self.encode_x), dtype=x.dtype)[0]

    def slots(self, page_table, sequence, positions):
        page = page_table[sequence, positions.long() // self.page_size].long()
        return page * self.page_size + positions.long() % self.page_size

    def __call__(self, x, positions, slots, page_table, lengths, q_starts=None, max_q=0):
        """x [T, hidden] of the sequences' last tokens -> [T, hidden], the cache written on the way."""
        H, K, D = self.heads, self.kv_heads, self.head_dim
        qkv = self.project(x, self.w_in, self.s_in).unflatten(1, (H + 2 * K, D))
        turned = qkv[:, : H + K]
        nv.rope(turned, positions, self.table, out=turned)  # queries and keys in one call, in place
        nv.kv_write(turned[:, H:], qkv[:, H + K:], self.cache, slots, encode_k=self.encode_k, encode_v=self.encode_v)
        self.queries = turned[:, :H]  # (kept for the comparison)
        y = nv.attention(self.queries, self.cache, page_table, lengths, q_starts=q_starts, max_q=max_q,
                         encode_k=self.encode_k, encode_v=self.encode_v)
        self.attended = y
        return self.project(y.flatten(1), self.w_out, self.s_out)

    def reference(self, queries, page_table, lengths, counts):
        """What attention gives in fp32 for these queries, from the values in the cache."""
        out, at = [], 0
        for b, (length, n) in enumerate(zip(lengths.tolist(), counts)):
            t = torch.arange(length, device=queries.device)
            k, v = nv.kv_read(self.cache, self.slots(page_table, b, t), encode_k=self.encode_k, encode_v=self.encode_v)
            q = queries[at: at + n].float().unflatten(1, (self.kv_heads, -1))
            score = torch.einsum("nhgd,thd->nhgt", q, k) / self.head_dim ** 0.5
            hidden = t > torch.arange(length - n, length, device=t.device).view(-1, 1, 1, 1)
            p = torch.softmax(score.masked_fill(hidden, -float("inf")), -1)
            out.append(torch.einsum("nhgt,thd->nhgd", p, v).flatten(1, 2))
            at += n
        return torch.cat(out)


def main(steps=8):
    dev = "cuda:0"
    layer = Layer()
    counts = [200, 37, 1, 129]
    B, T = len(counts), sum(counts)
    page_table = torch.randperm(64, device=dev)[: B * layer.max_pages].view(B, -1).int()
    lengths = torch.tensor(counts, dtype=torch.int32, device=dev)
    starts = torch.tensor([0] + counts, device=dev).cumsum(0).int()
    sequence = torch.repeat_interleave(torch.arange(B, device=dev), lengths)
    positions = torch.cat([torch.arange(n, device=dev) for n in counts]).int()
    x = torch.randn(T, 1024, device=dev).bfloat16()
    layer(x, positions, layer.slots(page_table, sequence, positions), page_table, lengths, starts, max(counts))
    want = layer.reference(layer.queries, page_table, lengths, counts)
    worst = ((layer.attended.float() - want).norm() / want.norm()).item()

    # single tokens: a step is captured once, its buffers filled anew each time
    x = torch.randn(B, 1024, device=dev).bfloat16()
    positions = lengths.clone()
    slots = layer.slots(page_table, torch.arange(B, device=dev), positions)
    lengths += 1
    layer(x, positions, slots, page_table, lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, positions, slots, page_table, lengths)
    for _ in range(steps):
        x.copy_(torch.randn(B, 1024, device=dev))
        graph.replay()
        want = layer.reference(layer.queries, page_table, lengths, [1] * B)
        worst = max(worst, ((layer.attended.float() - want).norm() / want.norm()).item())
        if not torch.isfinite(out).all():
            raise RuntimeError("an output is not finite")
        positions += 1
        lengths += 1
        slots.copy_(layer.slots(page_table, torch.arange(B, device=dev), positions))
    print(f"{T} prompt tokens and {steps} steps: attention off by {worst:.2e} of its norm from fp32 on the cache's values")
    return worst


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
