"""The example's layer against a model of it in 64 bits, step by step over several evictions: the
QKV product, rotation, cache contents, attention, weight sums, what an eviction keeps, and the
output product, as they run together."""
import numpy as np
import pytest

import oracle
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from gguf_block_quantized_q4_gb300.examples import decode_layer  # noqa: E402
from oracle import kv  # noqa: E402
from tests.kv_cases import numpy_of  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


@pytest.mark.parametrize("kind", [mq.Q8_0, mq.F16, mq.BF16])
def test_steps_and_evictions(kind):
    S, hq, hkv, dim, K, limit, keep = 3, 6, 2, 64, 256, 40, 21
    rows = (hq + 2 * hkv) * dim
    wqkv_raw = synth.weights(synth.Q4_K, rows, K, 1)
    wo_raw = synth.weights(synth.Q8_0, 128, hq * dim, 2)
    layer = decode_layer.DecodeLayer(
        mq.register_weight(mq.Q4_K, wqkv_raw, rows, K), mq.register_weight(mq.Q8_0, wo_raw, 128, hq * dim),
        S, hq, hkv, dim, limit, keep, sink=2, recent=5, kind=kind, page_size=7, max_pos=500,
        bias=torch.randn(rows, device="cuda"))
    bias = layer.bias.cpu().numpy()
    table = layer.rope.table.cpu().numpy()
    # the model's cache: rows of values per sequence, with the sums of their weights
    ks = [np.zeros((0, hkv, dim)) for _ in range(S)]
    vs = [np.zeros((0, hkv, dim)) for _ in range(S)]
    sums = [np.zeros((0, hkv)) for _ in range(S)]
    rng = np.random.default_rng(3)
    dtype = {mq.F16: torch.float16, mq.BF16: torch.bfloat16}.get(kind)
    for step in range(90):
        x = (rng.normal(size=(S, K)) * 0.02).astype(np.float32)
        evicted = len(layer.kept)
        y = layer.step(torch.from_numpy(x).cuda())
        mq.stream_status()
        for s, kept in layer.kept[evicted:]:  # the model keeps the rows that the device chose,
            kept = kept[0].cpu().numpy()      # after a look at the choice
            gathered = ks[s], vs[s], sums[s]
            new = [np.zeros((keep, *t.shape[1:])) for t in gathered]
            for h in range(hkv):
                worth = sums[s][:, h]
                chosen = kept[h]
                assert chosen[:2].tolist() == [0, 1] and chosen[-5:].tolist() == list(range(limit - 5, limit))
                assert (np.diff(chosen) > 0).all()
                inner = np.setdiff1d(np.arange(2, limit - 5), chosen)
                # (equal but for rounding where they differ)
                assert worth[chosen[2:-5]].min() >= worth[inner].max() * (1 - 1e-4)
                for t, n in zip(gathered, new):
                    n[:, h] = t[chosen, h]
            ks[s], vs[s], sums[s] = new
        # queries, keys and values in binary32 from the product's own output (checked elsewhere)
        qkv = mq.matvec(layer.wqkv, torch.from_numpy(x).cuda()).cpu().numpy() + bias
        qkv = qkv.reshape(S, -1, dim)
        pos = np.full((1, S), step)
        rot = kv.rope(qkv[:, :hq + hkv], table, pos, [0] * (dim // 2), False)
        out = np.zeros((S, hq, dim))
        for s in range(S):
            new = []
            for r in (rot[s, hq:], qkv[s, hq + hkv:]):
                if kind == mq.Q8_0:
                    q, d = kv.quantise_rows(r)
                    new.append(q.astype(np.float64) * np.repeat(d.astype(np.float64), 32, -1))
                else:
                    new.append(numpy_of(torch.from_numpy(r).to(dtype)).astype(np.float64))
            ks[s] = np.concatenate([ks[s], new[0][None]])
            vs[s] = np.concatenate([vs[s], new[1][None]])
            sums[s] = np.concatenate([sums[s], np.zeros((1, hkv))])
            assert len(ks[s]) == layer.held[s] <= limit
            for a in range(hq):
                h = a // (hq // hkv)
                w = ks[s][:, h] @ rot[s, a].astype(np.float64) * dim ** -0.5
                w = np.exp(w - w.max())
                w /= w.sum()
                out[s, a] = w @ vs[s][:, h]
                sums[s][:, h] += w
        # the output product of the model's attention: within the product's own bound, and what
        # the attention's error of 1e-5 of its largest value makes of it
        ref, bound = oracle.matvec(synth.Q8_0, wo_raw, 128, hq * dim, out.reshape(S, -1).astype(np.float32))
        slack = 1e-4 * bound + 1e-5 * np.abs(out).max() * bound / np.abs(out.reshape(S, -1)).mean(1, keepdims=True)
        assert (np.abs(y.cpu().numpy() - ref) <= slack + 1e-30).all(), step
    assert len(layer.kept) >= 2 * S


def test_the_example_runs(capsys):
    decode_layer.main(steps=300)
    out = capsys.readouterr().out
    assert "300 steps" in out and "as a graph" in out
