"""The paged cache's calls beside one another: strided page tables and planes, many sequences,
several streams, refused launches, and the order of calls on one stream without waits between."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from oracle import kv  # noqa: E402
from tests.kv_cases import Paged, attn_bound  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


def queries(S, hq, dim, seed):
    return torch.randn((S, hq, dim), generator=torch.Generator().manual_seed(seed))


def check(o, p, q, dim, lens=None):
    ref, mass, reach, _ = kv.attn_decode(p.host, p.page_size, q.numpy(), p.pages_host,
                                         lens or p.lens_list, dim ** -0.5)
    err = np.abs(o.cpu().numpy() - ref)
    assert (err <= attn_bound(dim, reach, mass, ref, "f32")).all()


@pytest.mark.parametrize("S", [33, 64, 1000, 3001])
def test_many_sequences(S):
    """More sequences than lanes, most of them short, some idle."""
    rng = np.random.default_rng(S)
    lens = [int(n) for n in rng.integers(0, 40, S)]
    lens[S // 2] = 700
    p = Paged("f16", lens, 1, 64, 16, seed=S)
    q = queries(S, 2, 64, S)
    check(mq.attn_decode(p.cache, q.cuda(), p.pages, p.lens, p.max_len), p, q, 64)
    mq.stream_status()


def test_strided_page_tables():
    p = Paged("f16", [100, 37], 2, 64, 16, seed=1, sums=True)
    q = queries(2, 4, 64, 2)
    wide = torch.full((2, p.pages.shape[1] + 13), 0x7FFFFFFF, dtype=torch.int32, device="cuda")
    wide[:, :p.pages.shape[1]] = p.pages
    view = wide[:, :p.pages.shape[1]]
    check(mq.attn_decode(p.cache, q.cuda(), view, p.lens, p.max_len), p, q, 64)
    new = torch.tensor(p.free[:2], dtype=torch.int32, device="cuda").view(2, 1)
    a = mq.kv_evict(p.cache, view, p.lens, p.max_len, new, 16)[0]
    assert torch.equal(a, mq.kv_evict(p.cache, p.pages, p.lens, p.max_len, new, 16)[0])
    with pytest.raises(ValueError):
        mq.attn_decode(p.cache, q.cuda(), wide.t(), p.lens, p.max_len)
    mq.stream_status()


def test_planes_with_gaps_between_pages():
    """A cache that is a slice of a larger allocation: the rows of several layers in one page."""
    p = Paged("q8_0", [100, 37], 2, 128, 16, seed=3)
    layered = {n: torch.full((t.shape[0], 3, *t.shape[1:]), 99, dtype=t.dtype, device="cuda")
               for n, t in p.dev.items()}
    for n, t in p.dev.items():
        layered[n][:, 1] = t
    v = {n: t[:, 1] for n, t in layered.items()}
    cache = mq.KVCache(mq.Q8_0, v["k"], v["v"], v["k_scale"], v["v_scale"])
    q = queries(2, 4, 128, 4)
    check(mq.attn_decode(cache, q.cuda(), p.pages, p.lens, p.max_len), p, q, 128)
    mq.stream_status()


def test_negative_scales():
    """Q8_0 scales of either sign stand for their values."""
    p = Paged("q8_0", [200], 1, 128, 16, seed=5)
    for n in ("k_scale", "v_scale"):
        flip = torch.rand(p.host[n].shape, generator=torch.Generator().manual_seed(6)).numpy() < 0.5
        p.host[n] = np.where(flip, -p.host[n], p.host[n])
        p.dev[n].copy_(torch.from_numpy(p.host[n]))
    q = queries(1, 3, 128, 7)
    check(mq.attn_decode(p.cache, q.cuda(), p.pages, p.lens, p.max_len), p, q, 128)


def test_scales_of_very_different_size():
    """Value scales from the smallest f16 to the largest, in one tile and from tile to tile."""
    p = Paged("q8_0", [600], 1, 64, 16, seed=8)
    e = torch.randint(-24, 16, p.host["v_scale"].shape, generator=torch.Generator().manual_seed(9))
    p.host["v_scale"] = np.where(np.isnan(p.host["v_scale"]), p.host["v_scale"],
                                 np.exp2(e.numpy()).astype(np.float16))
    p.dev["v_scale"].copy_(torch.from_numpy(p.host["v_scale"]))
    q = queries(1, 2, 64, 10)
    check(mq.attn_decode(p.cache, q.cuda(), p.pages, p.lens, p.max_len), p, q, 64)


def test_streams_side_by_side():
    """Two streams with a workspace each give the results of one after the other, bit for bit."""
    cases = []
    for i, (kind, lens) in enumerate((("f16", [3000, 5, 900]), ("q8_0", [2500, 1200]))):
        p = Paged(kind, lens, 2, 128, 16, seed=i)
        q = queries(len(lens), 8, 128, i).cuda()
        ws = mq.attn_workspace(p.cache, len(lens), 8, p.max_len)
        cases.append((p, q, ws, mq.attn_decode(p.cache, q, p.pages, p.lens, p.max_len, ws=ws)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    out = [[], []]
    for _ in range(20):
        for (p, q, ws, _), st, o in zip(cases, streams, out):
            with torch.cuda.stream(st):
                o.append(mq.attn_decode(p.cache, q, p.pages, p.lens, p.max_len, ws=ws))
    torch.cuda.synchronize()
    mq.stream_status()
    for (_, _, _, ref), o in zip(cases, out):
        assert all(torch.equal(x, ref) for x in o)


def test_store_attend_evict_without_waits():
    """Each call reads what the call before it wrote, on one stream: the same as with a wait after
    each."""
    results = []
    for wait in (True, False):
        g = torch.Generator(device="cuda").manual_seed(11)
        cache = mq.kv_cache(mq.F16, 40, 16, 2, 64, sums=True)
        rope = mq.Rope(mq.rope_table(400, [1e4 ** (-i / 32) for i in range(32)]))
        pages = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10)
        new = torch.arange(20, 30, dtype=torch.int32, device="cuda").view(2, 5)
        ws = mq.attn_workspace(cache, 2, 4, 160, track=True)
        outs = []

        def done(x):
            if wait:
                torch.cuda.synchronize()
            return x
        for t in range(120):
            qkv = torch.randn((2, 8 * 64), generator=g, device="cuda")
            pos = torch.full((1, 2), t, dtype=torch.int32, device="cuda")
            slot = pages[:, t // 16].long() * 16 + t % 16
            lens = torch.full((2,), t + 1, dtype=torch.int32, device="cuda")
            q = done(mq.rope_store(cache, rope, qkv, pos, slot, 4))
            outs.append(done(mq.attn_decode(cache, q, pages, lens, 160, track=True, ws=ws)))
        kept, lens = mq.kv_evict(cache, pages, lens, 160, new, 70, sink=2, recent=10)
        done(kept)
        outs.append(done(mq.attn_decode(cache, q, new, lens, 80, ws=ws)))
        torch.cuda.synchronize()
        mq.stream_status()
        results.append((outs, kept, cache.sums))
    (a, ka, sa), (b, kb, sb) = results
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(ka, kb) and torch.equal(sa, sb)


def test_refused_launches_are_reported(monkeypatch):
    p = Paged("f16", [100], 1, 64, 16, seed=12, sums=True)
    q = queries(1, 2, 64, 13).cuda()
    rope = mq.Rope(mq.rope_table(10, [1.0] * 32))
    new = torch.tensor([p.free[:1]], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    calls = {"attn_decode": lambda: mq.attn_decode(p.cache, q, p.pages, p.lens, 100),
             "evict_select": lambda: mq.kv_evict(p.cache, p.pages, p.lens, 100, new, 16),
             "rope_store": lambda: mq.rope_store(p.cache, rope, torch.zeros((1, 256), device="cuda"),
                                                 zero.int().view(1, 1), zero - 1, 2)}
    monkeypatch.setenv("MQ_TEST_FAIL_LAUNCH", "1")
    mq.init(0)
    try:
        for name, call in calls.items():
            with pytest.raises(mq.MQError, match=name) as e:
                call()
            assert e.value.name == "MQ_ERR_LAUNCH"
    finally:
        monkeypatch.delenv("MQ_TEST_FAIL_LAUNCH")
        mq.init(0)
    for call in calls.values():
        call()
    torch.cuda.synchronize()
    mq.stream_status()
