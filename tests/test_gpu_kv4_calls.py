"""Calls over a Q4_0 cache beside one another: captured and replayed, on two streams, in place, of sequences
that share pages, and with keys that are no numbers."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from oracle import kv  # noqa: E402
from tests.kv4_cases import Paged4  # noqa: E402
from tests.kv_cases import numpy_of  # noqa: E402
from tests.test_gpu_kv4 import check, queries  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_in_place(io):
    p = Paged4([300, 0, 33, 2000], 2, 128, 16, seed=1)
    q = queries(4, 14, 128, io, 2).cuda()
    want = mq.attn_decode(p.cache, q, p.pages, p.lens, p.max_len)
    o = q.clone()
    assert torch.equal(mq.attn_decode(p.cache, o, p.pages, p.lens, p.max_len, o=o), want)
    mq.stream_status()


@pytest.mark.parametrize("track", [False, True])
def test_replayed_with_other_lengths(track):
    """A captured call reads lengths, pages and queries of the time it is replayed; its workspace is ready
    again afterwards."""
    p = Paged4([900, 17, 256], 2, 64, 16, sums=True, seed=3)
    q = queries(3, 8, 64, "f32", 4).cuda()
    ws = mq.attn_workspace(p.cache, 3, 8, p.max_len, track=track)
    o = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            mq.attn_decode(p.cache, q, p.pages, p.lens, p.max_len, ws=ws, o=o, track=track)
    for lens in ([900, 17, 256], [1, 0, 200], [640, 5, 0]):
        p.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        q.mul_(0.9)
        sums = p.cache.sums.clone()
        graph.replay()
        torch.cuda.synchronize()
        got, after = o.clone(), p.cache.sums.clone()
        p.cache.sums.copy_(sums)
        want = mq.attn_decode(p.cache, q, p.pages, p.lens, p.max_len, track=track)
        assert torch.equal(got, want) and torch.equal(after.nan_to_num(), p.cache.sums.nan_to_num())
    mq.stream_status()


def test_two_streams():
    p = Paged4([3000, 100, 777], 4, 128, 32, seed=5)
    q = [queries(3, 28, 128, "f32", s).cuda() for s in (1, 2)]
    want = [mq.attn_decode(p.cache, x, p.pages, p.lens, p.max_len) for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [mq.attn_decode(p.cache, q[i % 2], p.pages, p.lens, p.max_len, stream=streams[i % 2]) for i in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % 2]) for i, o in enumerate(got))
    mq.stream_status()


def test_sequences_that_share_pages():
    """Several new tokens of a sequence: entries with the same pages and their own lengths."""
    p = Paged4([500], 2, 96, 24, seed=6)
    lens = [500, 499, 498, 24, 1, 0]
    p.pages = p.pages.repeat(6, 1).contiguous()
    p.pages_host, p.lens_list = np.repeat(p.pages_host, 6, 0), lens
    p.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    check(p, queries(6, 8, 96, "f32", 7), "f32", 96)


def test_keys_that_are_no_numbers():
    """A NaN among a key's scales makes its head's outputs NaN, and no other's."""
    p = Paged4([200, 60], 2, 128, 16, seed=8)
    page, slot = kv.place(p.pages_host[0], 16, np.array([150]))
    sc = p.host["k_scale"].copy()
    sc[page[0], 1, slot[0], 2] = np.nan
    p.set("k", kv.pack4((p.host["k"] + 8).astype(np.uint8)), sc)
    p.cache = p.wrap()
    q = queries(2, 6, 128, "f32", 9)
    o = mq.attn_decode(p.cache, q.cuda(), p.pages, p.lens, p.max_len)
    mq.stream_status()
    bad = torch.isnan(o).all(-1)
    assert bad.tolist() == [[False] * 3 + [True] * 3, [False] * 6]
    assert torch.isfinite(o[~bad]).all()


def test_rising_logits():
    """Logits that grow along the sequence by less and by more than the reference's slack, so that it is kept
    for some tiles and renewed at others."""
    n, dim = 3000, 64
    for total in (5.0, 60.0, 3000.0):
        p = Paged4([n], 1, dim, 16, seed=10)
        page, slot = kv.place(p.pages_host[0], 16, np.arange(n))
        packed = kv.pack4((p.host["k"] + 8).astype(np.uint8))
        sc = np.zeros_like(p.host["k_scale"])
        sc[:] = np.nan
        packed[page, 0, slot] = 0x99  # all numbers 1: the logit is the scale times the queries' sum
        sc[page, 0, slot] = (np.arange(n) / n)[:, None] * total / dim
        p.set("k", packed, sc.astype(np.float16))
        p.cache = p.wrap()
        q = torch.full((1, 4, dim), 1.0)
        q[0, 1] *= -1
        q[0, 2] *= 0.1
        q[0, 3, ::2] = 0
        check(p, q, "f32", dim, scale=1.0)


@pytest.mark.parametrize("dim", [64, 128])
def test_offsets_past_32_bits(dim):
    """Rows whose byte offsets pass 2^32: pages far apart in a strided plane."""
    S, n, hkv, ps = 2, 100, 1, 16
    small = Paged4([n] * S, hkv, dim, ps, seed=11)
    q = queries(S, 4, dim, "f32", 12).cuda()
    want = mq.attn_decode(small.cache, q, small.pages, small.lens, small.max_len)
    n_pages = small.cache.n_pages
    apart = (1 << 33) // (dim // 2) // n_pages  # rows from page to page
    apart -= apart % 16
    planes = {}
    for name, t in small.dev.items():
        width = t.shape[-1] if t.dim() == 4 else 1
        wide = torch.empty(n_pages * apart * width, dtype=t.dtype, device="cuda")
        view = wide.as_strided((n_pages, hkv, ps, width), (apart * width, ps * width, width, 1))
        view.copy_(t.view(view.shape))
        planes[name] = view
    cache = mq.KVCache(mq.Q4_0, planes["k"], planes["v"], planes["k_scale"], planes["v_scale"])
    assert torch.equal(mq.attn_decode(cache, q, small.pages, small.lens, small.max_len), want)
    mq.stream_status()
