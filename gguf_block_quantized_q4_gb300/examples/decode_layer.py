"""One attention layer of a decoding engine, from the library's calls: the QKV product on
quantised weights, rotation and store into a paged cache, attention over it, the output product;
and the cache brought back to a budget when a sequence has outgrown it.

    python -m gguf_block_quantized_q4_gb300.examples.decode_layer

runs a few hundred steps of a small batch on random Q4_K weights of the Qwen2.5-0.5B head layout
and prints the time of a step, launched call by call and replayed as a CUDA graph.
"""
from __future__ import annotations

import torch

import gguf_block_quantized_q4_gb300 as mq


class DecodeLayer:
    """Attention of `n_seqs` sequences that grow by a token per step.  wqkv: Weight of
    (n_heads + 2 n_kv_heads) head_dim rows, wo: Weight of n_heads head_dim columns.  A sequence
    that reaches `limit` cached tokens is brought down to `keep` of them (the first `sink`, the
    last `recent`, and those that have gathered the most attention)."""

    def __init__(self, wqkv, wo, n_seqs, n_heads, n_kv_heads, head_dim, limit, keep, sink=4,
                 recent=16, kind=mq.Q8_0, page_size=16, bias=None, max_pos=32768, freq_base=1e6):
        if not 0 < keep < limit:
            raise ValueError(f"keep={keep} must leave room below limit={limit}")
        if sink < 0 or recent < 0 or sink + recent > keep:
            raise ValueError(f"sink={sink} and recent={recent} are more than keep={keep}")
        self.wqkv, self.wo, self.n_heads, self.bias = wqkv, wo, n_heads, bias
        self.limit, self.keep, self.sink, self.recent = limit, keep, sink, recent
        self.width = -(-limit // page_size)
        spare = -(-keep // page_size)  # pages that one eviction needs at a time
        n_pages = n_seqs * self.width + spare
        self.cache = mq.kv_cache(kind, n_pages, page_size, n_kv_heads, head_dim, sums=True)
        half = head_dim // 2
        self.rope = mq.Rope(mq.rope_table(max_pos, [freq_base ** (-i / half) for i in range(half)]))
        self.ws = mq.attn_workspace(self.cache, n_seqs, n_heads, limit, track=True)
        self.free = list(range(n_pages))
        self.table = [[] for _ in range(n_seqs)]    # pages of each sequence
        self.held = [0] * n_seqs                    # cached tokens
        self.seen = 0                               # tokens so far: the next position
        self.pages = torch.zeros((n_seqs, self.width), dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
        self.pos = torch.zeros((1, n_seqs), dtype=torch.int32, device="cuda")
        self.slot = torch.zeros(n_seqs, dtype=torch.int64, device="cuda")
        self.kept = []                              # what the evictions kept, for a look

    def prepare(self):
        """Room for the next token of every sequence: evicts, takes pages, and writes the lengths,
        positions and slots that the device calls read."""
        ps = self.cache.page_size
        if self.seen == self.rope.table.shape[0]:
            raise ValueError(f"position {self.seen} is past the rotation's table")
        for s, n in enumerate(self.held):
            if n == self.limit:
                self._evict(s)
            if self.held[s] == len(self.table[s]) * ps:
                self.table[s].append(self.free.pop())
            self.held[s] += 1
        last = [n - 1 for n in self.held]
        rows = [t + [0] * (self.width - len(t)) for t in self.table]
        self.pages.copy_(torch.tensor(rows, dtype=torch.int32))
        self.lens.copy_(torch.tensor(self.held, dtype=torch.int32))
        self.pos.fill_(self.seen)
        self.slot.copy_(torch.tensor([t[i // ps] * ps + i % ps for t, i in zip(self.table, last)]))
        self.seen += 1

    def _evict(self, s):
        spare = -(-self.keep // self.cache.page_size)
        new = [self.free.pop() for _ in range(spare)]
        kept, _ = mq.kv_evict(self.cache, self.pages[s:s + 1], self.lens[s:s + 1], self.limit,
                              torch.tensor([new], dtype=torch.int32, device="cuda"), self.keep,
                              sink=self.sink, recent=self.recent)
        self.kept.append((s, kept))
        self.free += self.table[s]
        self.table[s], self.held[s] = new, self.keep

    def attend(self, x):
        """The layer's device calls on x [n_seqs][K]: only launches, fit for a CUDA graph."""
        qkv = mq.matvec(self.wqkv, x)
        q = mq.rope_store(self.cache, self.rope, qkv, self.pos, self.slot, self.n_heads, bias=self.bias)
        o = mq.attn_decode(self.cache, q, self.pages, self.lens, self.limit, track=True, ws=self.ws)
        return mq.matvec(self.wo, o.flatten(1))

    def step(self, x):
        self.prepare()
        return self.attend(x)


def _random_q4_k(n, k, gen):
    """Bytes of a random Q4_K tensor with weights of about 0.02."""
    import numpy as np
    blocks = gen.integers(0, 256, size=(n * k // 256, 144), dtype=np.uint8)
    blocks[:, 0:2] = np.frombuffer(np.float16(6e-5).tobytes(), np.uint8)
    blocks[:, 2:4] = np.frombuffer(np.float16(4e-4).tobytes(), np.uint8)
    return blocks.reshape(-1)


def main(steps=300, n_seqs=4, n_heads=14, n_kv_heads=2, head_dim=64, k=1024):
    import numpy as np
    gen = np.random.default_rng(0)
    mq.init(0)
    rows, cols = (n_heads + 2 * n_kv_heads) * head_dim, 1024
    wqkv = mq.register_weight(mq.Q4_K, _random_q4_k(rows, k, gen), rows, k, mq.REG_NO_MMQ_PLANE)
    # (the output product takes n_heads * head_dim = 896 columns: not a whole number of 256-element
    # blocks, so Q8_0)
    raw = np.zeros((cols * n_heads * head_dim // 32, 34), np.uint8)
    raw[:, 0:2] = np.frombuffer(np.float16(2e-4).tobytes(), np.uint8)
    raw[:, 2:] = gen.integers(0, 256, size=(raw.shape[0], 32), dtype=np.uint8)
    wo = mq.register_weight(mq.Q8_0, raw.reshape(-1), cols, n_heads * head_dim, mq.REG_NO_MMQ_PLANE)
    layer = DecodeLayer(wqkv, wo, n_seqs, n_heads, n_kv_heads, head_dim, limit=256, keep=128)
    x = torch.randn((n_seqs, k), device="cuda")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for i in range(steps):
        layer.prepare()
        if i == steps - 1:
            start.record()
        y = layer.attend(x)
        if i == steps - 1:
            end.record()
        x = torch.nn.functional.normalize(y, dim=1) * k ** 0.5
    torch.cuda.synchronize()
    mq.stream_status()
    print(f"{steps} steps, {len(layer.kept)} evictions, {layer.held[0]} tokens cached of {layer.seen}")
    print(f"one step, call by call: {start.elapsed_time(end) * 1e3:.1f} us")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        layer.attend(x)
        with torch.cuda.graph(graph, stream=side):
            layer.attend(x)
    torch.cuda.synchronize()
    graph.replay()
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"one step, as a graph: {start.elapsed_time(end) * 1e3 / 20:.1f} us")
    mq.stream_status()


if __name__ == "__main__":
    main()
