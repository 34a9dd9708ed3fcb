"""A decoding step's operators as they run together: QKV product, norms with the rotation and the store into
a Q4_0 cache, attention with weight sums, eviction, output product, LM head and sampling, against a
model in 64 bits; call by call and replayed as a graph."""
import math

import numpy as np
import pytest

import oracle
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from gguf_block_quantized_q4_gb300.examples import decode_layer, decode_step  # noqa: E402
from oracle import kv, sampling  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


def test_layer_with_norms_over_a_4_bit_cache():
    S, hq, hkv, dim, K, limit, keep = 3, 6, 2, 64, 256, 40, 21
    rows, m = (hq + 2 * hkv) * dim, hq + hkv
    wo_raw = synth.weights(synth.Q8_0, 128, hq * dim, 2)
    g = torch.Generator().manual_seed(1)
    wq, wk = (torch.rand(dim, generator=g) + 0.5 for _ in range(2))
    layer = decode_layer.DecodeLayer(
        mq.register_weight(mq.Q4_K, synth.weights(synth.Q4_K, rows, K, 1), rows, K),
        mq.register_weight(mq.Q8_0, wo_raw, 128, hq * dim), S, hq, hkv, dim, limit, keep, sink=2, recent=5,
        kind=mq.Q4_0, page_size=7, max_pos=500, norm=mq.HeadNorm(wq.cuda(), wk.cuda(), 1e-5))
    table = layer.rope.table.cpu().numpy()
    w_heads = np.concatenate([np.broadcast_to(wq.numpy(), (hq, dim)), np.broadcast_to(wk.numpy(), (hkv, dim))])
    ks, vs = ([np.zeros((0, hkv, dim)) for _ in range(S)] for _ in range(2))
    rng = np.random.default_rng(3)
    for step in range(90):
        x = torch.from_numpy((rng.normal(size=(S, K)) * 0.02).astype(np.float32)).cuda()
        evicted = len(layer.kept)
        y = layer.step(x)
        mq.stream_status()
        for s, kept in layer.kept[evicted:]:
            kept = kept[0].cpu().numpy()
            for cache in (ks, vs):
                cache[s] = np.stack([cache[s][kept[h], h] for h in range(hkv)], 1)
        qkv = mq.matvec(layer.wqkv, x).cpu().numpy().reshape(S, -1, dim)
        f = kv.head_scale(qkv[:, :m], np.float32(1e-5)).astype(np.float32)
        rot = kv.rope((qkv[:, :m] * f[..., None]) * w_heads, table, np.full((1, S), step), [0] * (dim // 2), False)
        out = np.zeros((S, hq, dim))
        for s in range(S):
            for cache, r in ((ks, rot[s, hq:]), (vs, qkv[s, m:])):
                n, d = kv.quantise_rows4(r)
                cache[s] = np.concatenate([cache[s], ((n - 8.0) * np.repeat(d.astype(np.float64), 32, -1))[None]])
            assert len(ks[s]) == layer.held[s] <= limit
            for a in range(hq):
                h = a // (hq // hkv)
                w = ks[s][:, h] @ rot[s, a].astype(np.float64) * dim ** -0.5
                w = np.exp(w - w.max())
                out[s, a] = w @ vs[s][:, h] / w.sum()
        # within the product's own bound, and what the attention's error of 1e-5 of its largest value (a factor
        # of the norm that is one last place off included) makes of it
        ref, bound = oracle.matvec(synth.Q8_0, wo_raw, 128, hq * dim, out.reshape(S, -1).astype(np.float32))
        slack = 1e-4 * bound + 1e-5 * np.abs(out).max() * bound / np.abs(out.reshape(S, -1)).mean(1, keepdims=True)
        assert (np.abs(y.cpu().numpy() - ref) <= slack + 1e-30).all(), step
    assert len(layer.kept) >= 2 * S


def test_steps_from_token_to_token():
    """The drawn tokens are those of the logits that the step returns, and come next; a replayed graph does
    what the calls do."""
    S, hq, hkv, dim, K, V = 4, 4, 2, 64, 256, 3000
    rows = (hq + 2 * hkv) * dim

    def make(size=1.0):
        g = torch.Generator().manual_seed(5)
        layers = [decode_layer.DecodeLayer(
            mq.register_weight(mq.Q4_K, synth.weights(synth.Q4_K, rows, K, 10 + i), rows, K),
            mq.register_weight(mq.Q4_K, synth.weights(synth.Q4_K, K, hq * dim, 20 + i), K, hq * dim), S, hq, hkv, dim,
            64, 32, kind=mq.Q4_0, norm=mq.HeadNorm(*(torch.rand(dim, generator=g).cuda() + 0.5 for _ in range(2))))
            for i in range(2)]
        return decode_step.DecodeStep(
            torch.randn((V, K), generator=g).cuda(), layers, mq.register_weight(mq.Q6_K, synth.weights(synth.Q6_K, V, K, 30), V, K),
            temperature=torch.tensor([0.0, 1.0, 2.0, 0.7], device="cuda") * size,
            top_k=torch.tensor([0, 50, 0, 0], dtype=torch.int32, device="cuda"),
            top_p=torch.tensor([1.0, 0.9, 0.8, 1.0], device="cuda"))
    size = float(make().step().std())  # (random weights: logits of hundreds)
    model, other = make(size), make(size)
    graph = None
    seen = set()
    for step in range(70):
        logits = model.step()
        mq.stream_status()
        for b in range(S):
            kw = {k: (int if k == "top_k" else float)(v[b]) for k, v in model.settings.items()}
            want, lp, margin = sampling.sample(logits[b].cpu().numpy(), float(model.u[b]), **kw)
            assert margin < 2.0 ** -24 or int(model.token[b]) == want
            seen.add(int(model.token[b]))
        # the same with the other's step as a graph
        other.prepare()
        other.u.copy_(model.u)
        if graph is None:
            side, first = torch.cuda.Stream(), other.token.clone()
            side.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.stream(side):
                with torch.cuda.graph(graph, stream=side):
                    other.decode()
            torch.cuda.current_stream().wait_stream(side)
            other.token.copy_(first)
        graph.replay()
        assert torch.equal(other.token, model.token) and torch.equal(other.logprob, model.logprob), step
    assert len(model.layers[0].kept) > 0 and len(seen) > 3


def test_the_example_runs(capsys):
    decode_step.main(steps=40)
    out = capsys.readouterr().out
    assert "40 steps" in out and "as a graph" in out


def test_a_sequence_without_a_token_goes_on(capsys):
    """Logits that are all NaN give token -1; the next step takes the first row of the embedding for it."""
    S, K, V, dim = 2, 256, 300, 64
    layer = decode_layer.DecodeLayer(
        mq.register_weight(mq.Q4_K, synth.weights(synth.Q4_K, 4 * dim, K, 10), 4 * dim, K),
        mq.register_weight(mq.Q8_0, synth.weights(synth.Q8_0, K, 2 * dim, 20), K, 2 * dim), S, 2, 1, dim, 64, 32, kind=mq.Q4_0)
    embedding = torch.randn((V, K), generator=torch.Generator().manual_seed(1)).cuda()
    embedding[7] = math.nan
    model = decode_step.DecodeStep(embedding, [layer], mq.register_weight(mq.Q6_K, synth.weights(synth.Q6_K, V, K, 30), V, K))
    model.token[1] = 7
    assert torch.isnan(model.step()[1]).all()
    assert int(model.token[1]) == -1 and float(model.logprob[1]) == -math.inf and int(model.token[0]) >= 0
    assert torch.equal(model.embedding.index_select(0, model.token.clamp(min=0))[1], embedding[0])
    model.step()
    mq.stream_status()
