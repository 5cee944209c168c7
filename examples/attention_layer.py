"""One attention layer with Q4_K weights, served: two prompts, a few tokens of
decoding, a beam fork and a compaction of the page pool.

    python examples/attention_layer.py

The layer's projections are the quantized products, its cache the paged one:
quantize -> qkv product -> rotary positions and append -> attention over the
pages -> quantize -> output product. A server keeps the page tables, lengths
and reference counts on the device and a free-list policy on the host; here the
host hands out pages in order.
"""

from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import quantized_decode_mat_amd as xq  # noqa: E402
import workloads as wl  # noqa: E402

DEV = "cuda"


class Layer:
    """hidden -> hidden, `heads` query and `kv_heads` key and value heads."""

    def __init__(self, hidden=1024, heads=8, kv_heads=2, dim=128, slots=4, pages=64, page=16, width=24, window=0,
                 sinks=0, seed=1):
        g = wl.rng(seed)
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, dim
        self.rows, self.page, self.window, self.sinks = (heads + 2 * kv_heads) * dim, page, window, sinks
        self.w_qkv = torch.from_numpy(wl.q4k_weights(self.rows, hidden, g).reshape(-1)).to(DEV)
        self.w_out = torch.from_numpy(wl.q4k_weights(hidden, heads * dim, g).reshape(-1)).to(DEV)
        # the weights are drawn without a norm's scale; this one keeps the scores moderate
        self.scale = 1e-4
        i = torch.arange(dim // 2, dtype=torch.float64, device=DEV)
        self.rope = xq.xq_rope_plan(10000.0 ** (-2.0 * i / dim), [dim // 2])
        shape = (pages, kv_heads, page, dim)
        self.kv = xq.xq_kv_cache(torch.zeros(shape, dtype=torch.bfloat16, device=DEV),
                                 torch.zeros(shape, dtype=torch.bfloat16, device=DEV))
        ints = dict(dtype=torch.int32, device=DEV)
        self.tables = torch.full((slots, width), -1, **ints)
        self.lens, self.refs = torch.zeros(slots, **ints), torch.zeros(pages, **ints)
        self.status = torch.zeros(2, **ints)
        need = xq.xq_attn_decode_workspace_bytes(slots, heads, self.kv, width * page, window, sinks)
        self.workspace = torch.zeros(max(need, xq.xq_cache_workspace_bytes(pages, slots)), dtype=torch.uint8, device=DEV)

    def product(self, w, x, n):
        """x [tokens, k] f32 times the Q4_K weights [n, k], f32."""
        m, k = x.shape
        xb = torch.empty(xq.xq_q8k_bytes(m, k), dtype=torch.uint8, device=DEV)
        xq.xq_quantize_q8k(xb, x, m, k)
        y = torch.empty(m, n, dtype=torch.float32, device=DEV)
        need = xq.xq_gemm_q4k_small_m_workspace_bytes(m, n, k)
        ws = torch.zeros(need, dtype=torch.uint8, device=DEV) if need else None
        xq.xq_gemm_q4k_small_m(y, w, xb, m, n, k, workspace=ws)
        return y

    def grow(self, slot, count):
        """Room for `count` more tokens of a sequence; their positions and cache slots."""
        lens, table = self.lens.tolist(), self.tables[slot].tolist()
        free = [p for p, r in enumerate(self.refs.tolist()) if r == 0]
        first = lens[slot]
        for i in range(-(-first // self.page), -(-(first + count) // self.page)):
            table[i] = free.pop(0)
            self.refs[table[i]] = 1
            self.tables[slot, i] = table[i]
        self.lens[slot] = first + count
        pos = list(range(first, first + count))
        return pos, [table[p // self.page] * self.page + p % self.page for p in pos]

    def append(self, x, slots_and_counts, io):
        pos, places = [], []
        for slot, count in slots_and_counts:
            p, s = self.grow(slot, count)
            pos += p
            places += s
        pos = torch.tensor([pos], dtype=torch.int32, device=DEV)
        places = torch.tensor(places, dtype=torch.int64, device=DEV)
        h, k = self.heads, self.kv_heads
        qkv = self.product(self.w_qkv, x, self.rows).view(len(x), h + 2 * k, self.dim)
        q = torch.empty(len(x), h, self.dim, dtype=io, device=DEV)
        xq.xq_rope_append(q, self.kv, qkv[:, :h], qkv[:, h:h + k], qkv[:, h + k:], pos, self.rope, places)
        return q, qkv, pos

    def prompt(self, x, slots_and_counts):
        """Prompts' tokens x [tokens, hidden], one after the other."""
        q, qkv, pos = self.append(x, slots_and_counts, torch.bfloat16)
        out = torch.empty_like(q)
        rows = torch.tensor([s for s, _ in slots_and_counts], device=DEV)
        counts = [0] + [c for _, c in slots_and_counts]
        starts = torch.tensor(counts, device=DEV).cumsum(0).int()
        xq.xq_attn_prefill(out, q, self.kv, self.tables[rows], self.lens[rows], starts, max(counts), self.scale,
                           window=self.window, sinks=self.sinks)
        return self.product(self.w_out, out.float().view(len(x), -1), self.hidden), out, q

    def step(self, x, slots):
        """One new token per sequence."""
        q, qkv, pos = self.append(x, [(s, 1) for s in slots], torch.float32)
        out = torch.empty_like(q)
        rows = torch.tensor(slots, device=DEV)
        xq.xq_attn_decode(out, q, self.kv, self.tables[rows], self.lens[rows], self.scale, window=self.window,
                          sinks=self.sinks, workspace=self.workspace)
        return self.product(self.w_out, out.view(len(x), -1), self.hidden), out, q

    def fork(self, parents, children):
        ints = dict(dtype=torch.int32, device=DEV)
        children = torch.tensor(children, **ints)
        xq.xq_cache_free(self.kv, self.refs, self.tables, self.lens, children)
        xq.xq_cache_fork(self.kv, self.refs, self.tables, self.lens, torch.tensor(parents, **ints), children,
                         self.status, workspace=self.workspace)

    def compact(self):
        xq.xq_cache_compact(self.kv, self.refs, self.tables, self.status, workspace=self.workspace)


def main():
    layer = Layer()
    g = torch.Generator(device=DEV).manual_seed(2)
    draw = lambda n: torch.randn(n, layer.hidden, device=DEV, generator=g)
    y, _, _ = layer.prompt(draw(70 + 33), [(0, 70), (1, 33)])
    print("prompts of 70 and 33 tokens ->", tuple(y.shape))
    for _ in range(3):
        y, _, _ = layer.step(draw(2), [0, 1])
    layer.fork([0, 0], [2, 3])
    print("two beams forked from the first, refused, lacking:", layer.status.tolist())
    for _ in range(3):
        y, _, _ = layer.step(draw(4), [0, 1, 2, 3])
    layer.fork([3], [1])
    layer.compact()
    print("live pages after the compaction:", layer.status.tolist()[1], "lengths:", layer.lens.tolist())
    y, _, _ = layer.step(draw(4), [0, 1, 2, 3])
    print("after it:", tuple(y.shape), "finite:", bool(y.isfinite().all()))


if __name__ == "__main__":
    main()
