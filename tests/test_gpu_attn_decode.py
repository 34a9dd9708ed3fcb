"""mq_attn_decode against the 64-bit definition, on caches whose unread rows and page entries are
poisoned."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from oracle import kv  # noqa: E402
from tests.kv_cases import IO, Paged, attn_bound, numpy_of  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


def queries(S, hq, dim, io, seed):
    g = torch.Generator().manual_seed(seed + 77)
    return (torch.randn((S, hq, dim), generator=g) * 1.5).to(IO[io])


def check(p, q, io, dim, window=0, track=False, scale=None, ws=None, stream=None):
    scale = dim ** -0.5 if scale is None else scale
    o = mq.attn_decode(p.cache, q.cuda(), p.pages, p.lens, p.max_len, scale=scale, window=window,
                       track=track, ws=ws)
    mq.stream_status()
    ref, mass, reach, weights = kv.attn_decode(p.host, p.page_size, numpy_of(q), p.pages_host,
                                               p.lens_list, scale, window)
    err = np.abs(numpy_of(o).astype(np.float64) - ref)
    bound = attn_bound(dim, reach, mass, ref, io)
    assert (err <= bound).all(), f"worst err/bound {np.max(err / bound):.3g}"
    if track:
        got = p.read("sums").astype(np.float64)
        want = p.host["sums"].astype(np.float64)
        slack = np.zeros_like(want)
        group = q.shape[1] // want.shape[1]
        for s, (lo, w) in enumerate(weights):
            if w.shape[1] == 0:
                continue
            page, slot = kv.place(p.pages_host[s], p.page_size, np.arange(lo, lo + w.shape[1]))
            rel = np.expm1(2 * reach[s].max() * (3 * dim / 16 + 2) * 2.0 ** -22 + 2.0 ** -17)
            for h in range(w.shape[0]):
                want[page, h, slot] += w[h]
                slack[page, h, slot] = w[h] * rel + np.abs(want[page, h, slot]) * 2.0 ** -22 + \
                    group * 1e-37
        live = ~np.isnan(want)
        assert np.array_equal(live, ~np.isnan(got))
        assert (np.abs(got - want)[live] <= slack[live]).all()
        p.host["sums"] = p.read("sums")
    return o


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200, 511, 513]


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_types_and_widths(kind, dim):
    p = Paged(kind, LENS, 2, dim, 16, seed=dim)
    check(p, queries(len(LENS), 8, dim, "f32", dim), "f32", dim)


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
def test_activation_types(kind, io):
    p = Paged(kind, [300, 0, 77, 1], 2, 128, 16, seed=3)
    check(p, queries(4, 14, 128, io, 4), io, 128)


@pytest.mark.parametrize("kind,dim", [("f16", 128), ("bf16", 64), ("q8_0", 96), ("f16", 256)])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (2, 1), (5, 1), (7, 1), (8, 1), (9, 1),
                                    (16, 1), (17, 1), (36, 2), (71, 1), (10, 5)])
def test_head_layouts(kind, dim, hq, hkv):
    p = Paged(kind, [130, 5, 0, 67], hkv, dim, 16, seed=hq)
    check(p, queries(4, hq, dim, "f32", hq), "f32", dim)


@pytest.mark.parametrize("page_size", [1, 3, 7, 16, 24, 64, 100, 1000])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_pages_and_layouts(page_size, layout):
    p = Paged("f16", [1, 130, 999, 24, 0], 3, 64, page_size, layout=layout, seed=page_size)
    check(p, queries(5, 6, 64, "f32", page_size), "f32", 64)
    p = Paged("q8_0", [1, 130, 999, 24, 0], 3, 128, page_size, layout=layout, seed=page_size + 1)
    check(p, queries(5, 6, 128, "f32", page_size), "f32", 128)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 511, 512, 5000])
@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
def test_sliding_window(kind, window):
    p = Paged(kind, LENS, 2, 128, 24, seed=window)
    check(p, queries(len(LENS), 4, 128, "f32", window), "f32", 128, window=window)


@pytest.mark.parametrize("kind,dim,hq,hkv", [("f16", 128, 28, 4), ("q8_0", 96, 12, 12),
                                             ("bf16", 64, 14, 2), ("f16", 256, 20, 1)])
@pytest.mark.parametrize("window", [0, 70])
def test_weight_sums(kind, dim, hq, hkv, window):
    """The sums grow by the attention weights, row by row, over two calls; rows outside the
    window or the lengths keep theirs."""
    p = Paged(kind, [0, 1, 17, 300, 64, 1025], hkv, dim, 16, sums=True, seed=hq)
    for seed in (1, 2):
        check(p, queries(6, hq, dim, "f32", seed), "f32", dim, window=window, track=True)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (5, 1), (6, 2), (12, 2), (9, 1), (12, 1),
                                    (17, 1), (23, 1), (33, 33), (80, 40)])
def test_weight_sums_of_all_group_sizes(hq, hkv):
    p = Paged("f16", [0, 700, 1, 129], hkv, 64, 24, sums=True, seed=hq)
    check(p, queries(4, hq, 64, "f32", hq), "f32", 64, track=True)
    check(p, queries(4, hq, 64, "f32", hq + 1), "f32", 64, window=33, track=True)


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("S,n", [(1, 20000), (3, 9000), (1, 50001)])
def test_long_sequences(kind, S, n):
    """Few rows, long: the length is split and joined."""
    p = Paged(kind, [n - 37 * i for i in range(S)], 2, 128, 64, seed=n, sums=True)
    check(p, queries(S, 14, 128, "f32", n), "f32", 128, track=True)


def test_many_unlike_sequences():
    rng = np.random.default_rng(5)
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(3000), 150))]
    lens[7] = 9000
    lens[8] = lens[149] = 0
    p = Paged("f16", lens, 2, 64, 16, seed=6)
    check(p, queries(150, 4, 64, "f32", 7), "f32", 64)


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
def test_uneven_weights(kind):
    """Logits over hundreds: all the weight on few keys, and the rest far below; also a scale of
    zero (all keys alike) and a negative one."""
    p = Paged(kind, [400, 33], 1, 128, 16, seed=8)
    q = queries(2, 4, 128, "f32", 9)
    check(p, q * 40, "f32", 128)
    check(p, q, "f32", 128, scale=0.0)
    check(p, q, "f32", 128, scale=-0.2)
    check(p, q * 1e-30, "f32", 128)
    check(p, torch.zeros_like(q), "f32", 128)


def test_the_first_keys_are_the_heaviest_and_the_last():
    """The running maximum falls behind at the start, or at the very end."""
    for at in (0, 299):
        p = Paged("f16", [300], 1, 128, 16, seed=10)
        q = queries(1, 2, 128, "f32", 11)
        page, slot = kv.place(p.pages_host[0], 16, np.array([at]))
        k = (q[0, 0] * 8).half()
        p.host["k"][page[0], 0, slot[0]] = k.numpy()
        p.dev["k"][page[0], 0, slot[0]] = k.cuda()
        check(p, q, "f32", 128)


def test_offsets_beyond_32_bits():
    """Rows more than 2^32 bytes and 2^31 elements into their plane."""
    n_pages, ps, dim = 3, 16, 128
    stride = 17 * (1 << 20) * ps // 16  # rows from page to page: 2 * 17 Mi rows of 256 bytes
    base = {n: torch.empty(2 * stride * dim + ps * dim, dtype=torch.float16, device="cuda")
            for n in ("k", "v")}
    view = {n: t.as_strided((n_pages, 1, ps, dim), (stride * dim, ps * dim, dim, 1))
            for n, t in base.items()}
    g = torch.Generator().manual_seed(1)
    host = {n: torch.randn((n_pages, 1, ps, dim), generator=g).half() for n in ("k", "v")}
    for n in ("k", "v"):
        view[n].copy_(host[n])
    cache = mq.KVCache(mq.F16, view["k"], view["v"])
    pages = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([40], dtype=torch.int32, device="cuda")
    q = queries(1, 2, dim, "f32", 2)
    o = mq.attn_decode(cache, q.cuda(), pages, lens, 48)
    mq.stream_status()
    ref, mass, reach, _ = kv.attn_decode({n: t.numpy() for n, t in host.items()}, ps, q.numpy(),
                                         pages.cpu().numpy(), [40], dim ** -0.5)
    err = np.abs(o.cpu().numpy() - ref)
    assert (err <= attn_bound(dim, reach, mass, ref, "f32")).all()


def test_one_workspace_for_calls_of_all_shapes():
    """A workspace kept over calls of other shapes, on its own stream: each call's result is that
    of a call with a fresh one, bit for bit."""
    big = Paged("f16", [5000, 7], 4, 128, 16, seed=1, sums=True)
    ws = mq.attn_workspace(big.cache, 64, 28, 5000, track=True)
    shapes = [("f16", [5000, 7], 4, 28, 128), ("q8_0", [3] * 40, 2, 14, 64),
              ("bf16", [1000] * 9, 1, 20, 256), ("f16", [4999], 1, 1, 96)]
    cases = []
    for i, (kind, lens, hkv, hq, dim) in enumerate(shapes):
        p = Paged(kind, lens, hkv, dim, 16, seed=i)
        q = queries(len(lens), hq, dim, "f32", i).cuda()
        cases.append((p, q, mq.attn_decode(p.cache, q, p.pages, p.lens, p.max_len)))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = []
    with torch.cuda.stream(st):
        for _ in range(3):
            for p, q, _ in cases:
                out.append(mq.attn_decode(p.cache, q, p.pages, p.lens, p.max_len, ws=ws))
    torch.cuda.synchronize()
    mq.stream_status()
    for i, o in enumerate(out):
        assert torch.equal(o, cases[i % len(cases)][2]), i


def test_graph_replay_follows_the_lengths():
    """Captured once for a bound, replayed as the sequences grow."""
    p = Paged("f16", [900, 40, 0], 2, 128, 16, seed=12)
    q = queries(3, 8, 128, "f32", 13)
    qd, lens = q.cuda(), p.lens.clone()
    ws = mq.attn_workspace(p.cache, 3, 8, p.max_len)
    o = torch.empty_like(qd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        mq.attn_decode(p.cache, qd, p.pages, lens, p.max_len, ws=ws, o=o)
        with torch.cuda.graph(g, stream=s):
            mq.attn_decode(p.cache, qd, p.pages, lens, p.max_len, ws=ws, o=o)
    for now in ([900, 40, 0], [3, 39, 0], [512, 1, 0], [0, 0, 0]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        ref, mass, reach, _ = kv.attn_decode(p.host, 16, q.numpy(), p.pages_host, now, 128 ** -0.5)
        err = np.abs(o.cpu().numpy() - ref)
        assert (err <= attn_bound(128, reach, mass, ref, "f32")).all(), now
    mq.stream_status()


def test_bad_lengths_and_pages_are_reported():
    """A length past the bound is clamped, a page outside the cache left out; the status says so
    once, and the other sequences are as they should be."""
    p = Paged("f16", [40, 20], 1, 64, 16, seed=14)
    q = queries(2, 2, 64, "f32", 15)
    good = mq.attn_decode(p.cache, q.cuda(), p.pages, p.lens, p.max_len)
    lens = torch.tensor([40, -3], dtype=torch.int32, device="cuda")
    o = mq.attn_decode(p.cache, q.cuda(), p.pages, lens, p.max_len)
    with pytest.raises(mq.MQError, match="length -3") as e:
        mq.stream_status()
    assert e.value.name == "MQ_ERR_INDEX"
    mq.stream_status()
    assert torch.equal(o[0], good[0]) and not o[1].any()
    for bad in (-1, 1 << 30):
        pages = p.pages.clone()
        pages[0, 1] = bad  # positions 16..31 of the first sequence
        o = mq.attn_decode(p.cache, q.cuda(), pages, p.lens, p.max_len)
        with pytest.raises(mq.MQError, match="page"):
            mq.stream_status()
        assert torch.equal(o[1], good[1])
        host = {n: t[p.pages_host[0, [0, 2]]] for n, t in p.host.items()}
        host = {n: np.concatenate([t[:1], t[1:]]) for n, t in host.items()}
        ref, mass, reach, _ = kv.attn_decode(host, 16, q.numpy()[:1], np.array([[0, 1]]), [24],
                                             64 ** -0.5)
        err = np.abs(o.cpu().numpy()[:1] - ref)
        assert (err <= attn_bound(64, reach, mass, ref, "f32")).all()


def test_refusals_on_the_device():
    p = Paged("f16", [40], 1, 64, 16, seed=16)
    q = queries(1, 2, 64, "f32", 17).cuda()
    with pytest.raises(mq.MQError) as e:
        mq.attn_decode(p.cache, q, p.pages, p.lens, p.max_len, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.name == "MQ_ERR_ARG" and "ws_bytes" in str(e.value)
    L = mq.lib()
    ws = mq.attn_workspace(p.cache, 1, 2, 40)

    def call(q_ptr, o_ptr, ws_ptr=None):
        return mq.STATUS[L.mq_attn_decode(p.cache._ref, 0, q_ptr, o_ptr, p.pages.data_ptr(), 3,
                                          p.lens.data_ptr(), 1, 2, 40, 0.1, 0, 0,
                                          ws_ptr or ws.data_ptr(), ws.numel(), None)]
    o = torch.empty_like(q)
    assert call(q.data_ptr(), o.data_ptr()) == "MQ_OK"
    assert call(None, o.data_ptr()) == "MQ_ERR_ARG"
    assert call(q.data_ptr() + 4, o.data_ptr()) == "MQ_ERR_ALIGN"
    assert call(q.cpu().data_ptr(), o.data_ptr()) == "MQ_ERR_ARG"
    assert call(q.data_ptr(), o.data_ptr(), ws.data_ptr() + 16) == "MQ_ERR_ALIGN"
    # no sequences: nothing to do
    assert mq.attn_decode(p.cache, q[:0], p.pages[:0], p.lens[:0], 40, ws=ws).shape == (0, 2, 64)
    torch.cuda.synchronize()
    mq.stream_status()
