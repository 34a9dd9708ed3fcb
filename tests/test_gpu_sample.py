"""mq_sample against the 64-bit definition: every token equal, but where a running sum lies so near a
border that 2^-24 of the sum decides."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from oracle.sampling import sample  # noqa: E402
from tests.kv_cases import IO, numpy_of  # noqa: E402

# A weight is right to 2^-27 of itself down to 2^-8 of the largest, so running sums and shares of those to 2^-26
# of the sum.  Below that it is right to 2^-21 with errors of either sign (mean -8e-9, 2^-27): 64 unlike
# logits or more leave 2^-21 / 8 of their share at most but rarely.  Rounding to units of 2^-44 (2^-38 or 2^-34
# in flat rows) adds half a unit of either sign a token, 2^-35 * sqrt(2^19) < 2^-25 in all; tokens below half a
# unit, at most 2^19 of them, add nothing where they should add up to 2^-26.
NEAR = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


def check(x, u, near=0.2, **given):
    """x [B][V] on the CPU; given: temperature, top_k, top_p, min_p as lists or None.  `near`: the share
    of rows that may lie near a border."""
    B = x.shape[0]
    dev = {k: None if v is None else torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32).cuda()
           for k, v in given.items()}
    u = torch.as_tensor(u, dtype=torch.float32)
    token, logprob = mq.sample(x.cuda(), u.cuda(), **dev)
    mq.stream_status()
    rows, skipped = numpy_of(x), 0
    host = {k: None if v is None else v.cpu().double().tolist() for k, v in dev.items()}
    for b in range(B):
        kw = {k: (int(v[b]) if k == "top_k" else v[b]) for k, v in host.items() if v is not None}
        want, lp, margin = sample(rows[b], float(u[b]), **kw)
        if margin < NEAR:
            skipped += 1
            continue
        assert int(token[b]) == want, (b, int(token[b]), want, margin, kw)
        # two quotients, a logarithm and a difference, each within 2^-23 of terms of this size; the sum's 2^-26
        assert np.isclose(float(logprob[b]), lp, rtol=2.0 ** -20, atol=2.0 ** -24), (b, float(logprob[b]), lp)
    assert skipped <= near * B
    return token, logprob


def rows(B, V, seed, io="f32", size=2.0, peaks=8):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, V), generator=g) * size
    at = torch.randint(0, V, (B, peaks), generator=g)
    x.scatter_(1, at, torch.rand((B, peaks), generator=g) * 6 * size + size)
    return x.to(IO[io]), torch.rand(B, generator=g)


VOCABS = [1, 2, 3, 5, 31, 32, 33, 255, 1000, 2047, 4099, 32003]


@pytest.mark.parametrize("V", VOCABS)
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_all_limits_at_once(V, io):
    B = 40
    x, u = rows(B, V, V, io)
    g = np.random.default_rng(V)
    check(x, u, temperature=(0.2 + g.random(B) * 2).tolist(), top_k=g.integers(-1, min(V, 300) + 2, B).tolist(),
          top_p=(g.random(B) * 1.2).tolist(), min_p=(g.random(B) * 0.3 - 0.1).tolist())


@pytest.mark.parametrize("V", [7, 1000, 32003, 151936])
@pytest.mark.parametrize("which", ["none", "k", "p", "m", "kp", "pm"])
def test_each_limit_alone(V, which):
    B = 12
    x, u = rows(B, V, V + 1)
    g = np.random.default_rng(V)
    check(x, u, near=0.5, temperature=(0.3 + g.random(B)).tolist(),
          top_k=g.integers(1, min(V, 5000), B).tolist() if "k" in which else None,
          top_p=g.random(B).tolist() if "p" in which else None,
          min_p=(g.random(B) * 0.1).tolist() if "m" in which else None)


@pytest.mark.parametrize("B,V", [(1, 151936), (1, 1), (1, 4096), (3, 300001), (300, 1234), (1, 524287), (2, 65536)])
def test_sizes(B, V):
    """One row over a whole cluster, more rows than blocks are resident, the largest vocabulary."""
    x, u = rows(B, V, B + V)
    check(x, u, near=1.0 if B < 4 else 0.2, temperature=[0.8] * B, top_k=[50] * B, top_p=[0.9] * B)
    check(x, u, near=1.0 if B < 4 else 0.2, temperature=[0.5] * B)


@pytest.mark.parametrize("V", [100, 5000, 40000])
@pytest.mark.parametrize("values", [1, 2, 7])
def test_many_equal_logits(V, values):
    """Cuts that fall among thousands of equal logits: the ones of lower index stay."""
    g = np.random.default_rng(V + values)
    B = 24
    x = torch.from_numpy(g.integers(0, values, (B, V)).astype(np.float32) * 0.5)
    k = g.integers(1, V + 1, B).tolist()
    check(x, g.random(B).astype(np.float32), near=0.3, top_k=k)
    # shares that no running sum of equal weights ends at
    p = [(i + 0.37) / V for i in g.integers(0, V, B)]
    check(x, g.random(B).astype(np.float32), near=0.3, top_p=p)
    check(x, g.random(B).astype(np.float32), near=0.3, top_k=k, top_p=p, min_p=[0.7] * B)


@pytest.mark.parametrize("V", [3000, 50000])
def test_nearly_equal_logits(V):
    """More tokens in one bin than a list holds, all of them unlike: cut by the logits' bits."""
    g = np.random.default_rng(V)
    B = 16
    x = torch.from_numpy((3 + g.random((B, V)) * 0.01).astype(np.float32))
    u = g.random(B).astype(np.float32)
    check(x, u, near=0.3, top_k=g.integers(1, V, B).tolist())
    check(x, u, near=0.3, top_p=g.random(B).tolist())
    check(x, u, near=0.3, top_k=g.integers(V // 2, V, B).tolist(), top_p=g.random(B).tolist())
    check(-x, u, near=0.3, top_k=g.integers(V // 2, V, B).tolist(), top_p=g.random(B).tolist())


def test_greedy_rows():
    x, u = rows(30, 5001, 3, "bf16")
    x = (x * 2).round() / 2  # ties
    token, logprob = check(x, u, temperature=[0.0, -1.0, float("nan")] * 10, top_k=[5] * 30, top_p=[0.5] * 30)
    first = [int((x[b].float() == x[b].float().max()).nonzero()[0]) for b in range(30)]
    assert token.tolist() == first and not logprob.any()


def test_masked_rows():
    """Tokens at minus infinity, at the type's lowest value and NaN; rows of which one or none is left."""
    for io in ("f32", "f16", "bf16"):
        x, u = rows(60, 3001, 4, io)
        g = torch.Generator().manual_seed(5)
        gone = torch.rand(x.shape, generator=g) < 0.99
        low = torch.tensor([-float("inf"), torch.finfo(IO[io]).min, float("nan")]).repeat(20)[:, None].to(IO[io])
        x = torch.where(gone, low, x)
        x[3], x[5] = -float("inf"), float("nan")
        x[6] = -float("inf")
        x[6, 2000] = -5.0
        x[7] = torch.finfo(IO[io]).min
        token, logprob = check(x, u, temperature=[0.9] * 60, top_k=[0, 40] * 30, top_p=[1.0, 0.8, 0.3] * 20, min_p=[0.0, 0.05] * 30)
        assert token[[3, 5, 6]].tolist() == [-1, -1, 2000] and logprob[3] == -float("inf")
        greedy, _ = mq.sample(x.cuda(), u.cuda(), temperature=torch.zeros(60, device="cuda"))
        assert greedy[[3, 5, 6, 7]].tolist() == [-1, -1, 2000, 0]


def test_infinite_logits_and_odd_settings():
    inf, nan = float("inf"), float("nan")
    x = torch.randn((12, 700))
    x[0, [5, 600]] = inf
    x[1, 3] = inf
    u = [0.7, 0.2, 1.0, 2.0, -1.0, nan, 0.0, 0.5, 0.5, 0.5, 0.5, 0.99]
    token, _ = check(x, u, temperature=[1, 1, 1, 1, 1, 1, 1, inf, 1e-40, 1e30, 3e38, inf], top_p=[1, 1, nan, 1, 1, 1, -1, 1, 1, 0.5, 1, 1],
                     min_p=[0, 0, nan, 0, 0, 0, 0, 2.0, 0, 0, 0.5, 0.5], top_k=[0, 1, -5, 0, 0, 0, 0, 0, 0, 700, 699, 1 << 30], near=0.4)
    assert token[:2].tolist() == [600, 3] and token[4] == token[5] == 0


def test_large_and_small_logits():
    g = np.random.default_rng(1)
    for size in (1e30, 1e5, 1e-3, 1e-30):
        x = torch.from_numpy((g.standard_normal((20, 999)) * size).astype(np.float32))
        check(x, g.random(20).astype(np.float32), temperature=[size * 0.5] * 20, top_p=[0.9] * 20, near=0.3)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shift,ld", [(1, 1003), (3, 1009), (0, 1001), (7, 1024)])
def test_rows_at_any_place(io, shift, ld):
    """Rows that start inside a 16-byte block, with neighbours that must not be drawn."""
    B, V = 9, 1000
    x, u = rows(B, V, 8, io)
    wide = torch.full((B * ld + 16,), 100.0, dtype=IO[io]).cuda()
    view = wide[shift:shift + B * ld].view(B, ld)[:, :V]
    view.copy_(x)
    want = mq.sample(x.cuda(), u.cuda(), top_k=torch.full((B,), 20, dtype=torch.int32, device="cuda"))
    got = mq.sample(view, u.cuda(), top_k=torch.full((B,), 20, dtype=torch.int32, device="cuda"))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check(view.cpu(), u, top_k=[20] * B)


def test_the_same_whatever_runs_beside():
    """The rows' results alone, in a batch (other cluster sizes), again, on another stream, in a graph."""
    B, V = 20, 100003
    x, u = rows(B, V, 9)
    x, u = x.cuda(), u.cuda()
    kw = dict(temperature=torch.linspace(0.5, 2.0, B, device="cuda"), top_p=torch.linspace(0.3, 0.99, B, device="cuda"))
    want = mq.sample(x, u, **kw)
    for b in (0, 7, 19):
        one = mq.sample(x[b:b + 1], u[b:b + 1], **{k: v[b:b + 1] for k, v in kw.items()})
        assert one[0] == want[0][b] and one[1] == want[1][b]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [mq.sample(x, u, stream=side, **kw) for _ in range(3)] + [mq.sample(x, u, **kw) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(g[0], want[0]) and torch.equal(g[1], want[1]) for g in got)
    token, logprob = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            mq.sample(x, u, token=token, logprob=logprob, **kw)
    for _ in range(2):
        token.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(token, want[0]) and torch.equal(logprob, want[1])
    u.copy_(1 - u)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(token, mq.sample(x, u, **kw)[0])
    mq.stream_status()


def test_draws_follow_the_shares():
    """Evenly spaced numbers give each token its share of them."""
    x = torch.log(torch.tensor([4.0, 1.0, 2.0, 1.0])).repeat(8000, 1).cuda()
    token, logprob = mq.sample(x, (torch.arange(8000, device="cuda") + 0.5) / 8000)
    assert torch.bincount(token.long(), minlength=4).tolist() == [4000, 1000, 2000, 1000]
    assert (token[1:] >= token[:-1]).all()
    none = mq.sample(x[:0], x[:0, 0])
    assert none[0].shape == (0,)


@pytest.mark.parametrize("down", [6.0, 9.0, 14.4, 20.0, 30.0])
@pytest.mark.parametrize("V", [2049, 151936])
def test_one_token_above_equal_ones(V, down):
    """All other tokens 2^-down of the first: their errors are all alike.  An exponential's 2^-21, and half a unit of
    2^-44 of the largest each (of 2^-38 or 2^-34 in flat rows: less than 2^-20 of the sum over 2^19 tokens, the
    second only where the sum is above 2^-15 of their number): 2^-19 in a place or a share."""
    bound = 2.0 ** -19
    B = 16
    l = torch.full((B, V), -down * math.log(2.0))
    l[:, V // 3] = 0.0
    u = (torch.arange(B) + 0.5) / B
    token, logprob = mq.sample(l.cuda(), u.cuda())
    mq.stream_status()
    w = np.exp(numpy_of(l)[0].astype(np.float64))
    run = np.cumsum(w) / w.sum()
    for b in range(B):
        i = int(token[b])
        before = run[i - 1] if i else 0.0
        assert before - bound <= float(u[b]) <= run[i] + bound, (b, i)
        # (a difference of logits, a logarithm and their sum are rounded to binary32 below 2^5)
        assert abs(float(logprob[b]) - math.log(w[i] / w.sum())) < 2 * bound + 3 * 2.0 ** -20


def test_logits_on_the_host_are_refused():
    with pytest.raises(mq.MQError, match="logits"):
        mq.sample(torch.zeros((2, 50)), torch.zeros(2, device="cuda"))


@pytest.mark.parametrize("B", [64, 300, 512, 513])
def test_many_rows_of_unlike_settings(B):
    """More rows than are resident at once, whatever the order they are taken in: each has its own answer."""
    g = torch.Generator().manual_seed(B)
    V = 20000
    x = torch.randn((B, V), generator=g) * 2

    def pick(*values):
        return [values[int(i)] for i in torch.randint(0, len(values), (B,), generator=g)]
    given = dict(temperature=pick(0.0, 0.7, 1.5), top_k=pick(0, 0, 20, 900, V), top_p=pick(1.0, 0.6, 0.95),
                 min_p=pick(0.0, 0.0, 0.05))
    u = torch.rand(B, generator=g)
    check(x, u, **given)
    alike = {k: [v[0]] * B for k, v in given.items()}
    alike["top_p"], alike["temperature"] = [0.8] * B, [1.0] * B
    check(x[:64], u[:64], **{k: v[:64] for k, v in alike.items()})
