"""mq_sample: a row's answer is the same wherever its logits lie, in all calls alike, and the definition's for single rows
of every size."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from oracle.sampling import sample as exact  # noqa: E402
from tests.kv_cases import IO, numpy_of  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


def rows(B, V, seed, io="f32", size=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, V), generator=g) * size).to(IO[io]), torch.rand(B, generator=g)


def on_device(kw):
    return {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32).cuda() for k, v in kw.items()}


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("down", [7.2, 7.9, 15.0, 15.9])
def test_unit_does_not_depend_on_the_address(io, down):
    """Heavy tokens at both ends of every second group of 128, so that groups counted from an aligned address instead of
    the row's start would have another mean."""
    B, V, ln2 = 6, 20000, math.log(2)
    x = torch.full((B, V), -36 * ln2 if down < 8 else -40 * ln2)
    x[:, 0::256] = x[:, 127::256] = -down * ln2
    x[:, 7] = 0
    x[2, 100:4000] = -math.inf
    x = x.to(IO[io])
    u = torch.rand(B, generator=torch.Generator().manual_seed(1)).cuda()
    for kw in ({}, {"top_p": [0.999] * B}, {"temperature": [0.5, 1, 2, 1, 1, 0.7]}):
        given = on_device(kw)
        want = None
        for shift in range(8):
            for ld in (V, V + 1, V + 3):
                wide = torch.full((B * ld + 16,), 50.0, dtype=IO[io], device="cuda")
                view = wide[shift:shift + B * ld].view(B, ld)[:, :V]
                view.copy_(x)
                got = mq.sample(view, u, **given)
                want = want or got
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (kw, shift, ld)
    mq.stream_status()


@pytest.mark.parametrize("V", [32003, 100003])
def test_rows_of_an_odd_batch(V):
    """Contiguous rows of an odd length, each at another alignment: as alone."""
    B = 12
    x, u = rows(B, V, V)
    x, u = x.cuda(), u.cuda()
    for temperature in (0.3, 0.55, 0.8, 1.2):
        t = torch.full((B,), temperature, device="cuda")
        want = mq.sample(x, u, temperature=t)
        for b in range(B):
            one = mq.sample(x[b].clone()[None], u[b:b + 1], temperature=t[:1])
            assert one[0] == want[0][b] and one[1] == want[1][b], (temperature, b)
    mq.stream_status()


@pytest.mark.parametrize("k", [257, 289, 321, 353, 700, 1500])
def test_long_lists(k):
    """More tokens than are drawn from by counting, many rows and calls at once: one answer each."""
    B, V = 64, 30011
    x, u = rows(B, V, k)
    kw = {"top_k": [k] * B}
    given = on_device(kw)
    xd, ud = x.cuda(), u.cuda()
    got = [mq.sample(xd, ud, **given) for _ in range(20)]
    mq.stream_status()
    assert all(torch.equal(g[0], got[0][0]) and torch.equal(g[1], got[0][1]) for g in got)
    compared = 0
    for b in range(B):
        want, lp, margin = exact(numpy_of(x)[b], float(u[b]), top_k=k)
        if margin > 2.0 ** -24:
            compared += 1
            assert int(got[0][0][b]) == want and abs(float(got[0][1][b]) - lp) < 2.0 ** -18
    assert compared > B // 2


@pytest.mark.parametrize("B,V", [(1, 16384), (1, 151936), (2, 65536), (3, 300001), (1, 524287)])
@pytest.mark.parametrize("which", ["temperature", "top_p", "top_k", "min_p"])
def test_few_rows_of_every_size(B, V, which):
    """Every row is compared: with another number where the first lies next to a border."""
    x, u = rows(B, V, B + V)
    kw = {"temperature": [0.7] * B}
    if which != "temperature":
        kw[which] = [{"top_p": 0.9, "top_k": 50, "min_p": 0.01}[which]] * B
    given, xd = on_device(kw), x.cuda()
    open_rows = set(range(B))
    for attempt in range(12):
        got = [mq.sample(xd, u.cuda(), **given) for _ in range(4)]
        assert all(torch.equal(g[0], got[0][0]) and torch.equal(g[1], got[0][1]) for g in got)
        for b in range(B):
            want, lp, margin = exact(numpy_of(x)[b], float(u[b]), **{k: v[b] for k, v in kw.items()})
            if margin > 2.0 ** -24:
                open_rows.discard(b)
                assert int(got[0][0][b]) == want, (b, attempt)
                assert np.isclose(float(got[0][1][b]), lp, rtol=2.0 ** -20, atol=2.0 ** -24)
        u = torch.rand(B, generator=torch.Generator().manual_seed(100 + attempt))
    mq.stream_status()
    assert not open_rows
