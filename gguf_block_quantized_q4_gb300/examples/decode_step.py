"""Steps of a decoding engine from a token to the next one, from the library's calls: attention layers
with normed heads over a 4-bit cache, the LM head's product and sampling.

    python -m gguf_block_quantized_q4_gb300.examples.decode_step

runs a small batch on random weights and prints the time of a step replayed as a CUDA graph.
"""
from __future__ import annotations

import torch

import gguf_block_quantized_q4_gb300 as mq

from .decode_layer import DecodeLayer, _random_q4_k


class DecodeStep:
    """Layers (DecodeLayer, of the same sequences) between an embedding f32 [vocabulary][K] and an LM head
    (Weight of as many rows); the requests' settings as mq.sample takes them, one per sequence."""

    def __init__(self, embedding, layers, head, **settings):
        if not layers:
            raise ValueError("a step needs layers")
        if head.N != embedding.shape[0]:  # (a token without a row would be read past the embedding's end)
            raise ValueError(f"the head's {head.N} rows are not the embedding's {embedding.shape[0]}")
        if len({len(layer.held) for layer in layers}) > 1:
            raise ValueError("the layers are of unlike numbers of sequences")
        self.embedding, self.layers, self.head, self.settings = embedding, layers, head, settings
        n = len(layers[0].held)
        self.token = torch.zeros(n, dtype=torch.int32, device="cuda")    # the last ones, and their logprobs
        self.logprob = torch.zeros(n, dtype=torch.float32, device="cuda")
        self.u = torch.zeros(n, dtype=torch.float32, device="cuda")

    def prepare(self):
        """Room for the next token in every layer, and its random numbers."""
        for layer in self.layers:
            layer.prepare()
        self.u.uniform_()

    def decode(self):
        """The step's device calls, from self.token to the next one: only launches, fit for a CUDA
        graph."""
        x = self.embedding.index_select(0, self.token.clamp(min=0))  # (-1: a row whose logits were no numbers)
        for layer in self.layers:
            x = x + layer.attend(x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6))
        logits = mq.matvec(self.head, x)
        mq.sample(logits, self.u, token=self.token, logprob=self.logprob, **self.settings)
        return logits

    def step(self):
        self.prepare()
        return self.decode()


def main(steps=100, n_seqs=4, n_layers=2, n_heads=16, n_kv_heads=8, head_dim=128, k=1024, vocab=32000):
    import numpy as np
    gen = np.random.default_rng(0)
    mq.init(0)
    rows = (n_heads + 2 * n_kv_heads) * head_dim

    def weight(n, columns):
        return mq.register_weight(mq.Q4_K, _random_q4_k(n, columns, gen), n, columns, mq.REG_NO_MMQ_PLANE)

    def norm():
        return mq.HeadNorm(*(1 + 0.1 * torch.randn(head_dim, device="cuda") for _ in range(2)))
    layers = [DecodeLayer(weight(rows, k), weight(k, n_heads * head_dim), n_seqs, n_heads, n_kv_heads, head_dim,
                          limit=256, keep=128, kind=mq.Q4_0, norm=norm()) for _ in range(n_layers)]

    def row(*values, dtype=torch.float32):
        return torch.tensor((values * n_seqs)[:n_seqs], dtype=dtype, device="cuda")
    model = DecodeStep(torch.randn((vocab, k), device="cuda"), layers, weight(vocab, k),
                       temperature=row(0.0, 0.7, 1.0), top_k=row(0, 40, 0, dtype=torch.int32), top_p=row(1.0, 0.95, 0.9),
                       min_p=row(0.0, 0.0, 0.02))
    for _ in range(steps):
        model.step()
    torch.cuda.synchronize()
    mq.stream_status()
    print(f"{steps} steps; the last tokens {model.token.tolist()}, their logprobs "
          f"{[round(v, 2) for v in model.logprob.tolist()]}")
    model.prepare()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        model.decode()
        with torch.cuda.graph(graph, stream=side):
            model.decode()
    torch.cuda.synchronize()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    graph.replay()
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"one step of {n_layers} layers, as a graph: {start.elapsed_time(end) * 1e3 / 20:.1f} us")
    mq.stream_status()


if __name__ == "__main__":
    main()
