"""mq_kv_evict: the rows that stay, their order and their copies against the definition, exactly."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from oracle import kv  # noqa: E402
from tests.kv_cases import Paged  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


def bits(a):
    return np.ascontiguousarray(a).view({1: np.uint8, 2: np.uint16, 4: np.uint32}[a.dtype.itemsize])


def check(p, keep, sink=0, recent=0, sums=None):
    """Evicts into the cache's spare pages and compares every plane, row by row."""
    S, hkv = len(p.lens_list), p.cache.n_kv_heads
    if sums is not None:
        p.host["sums"] = sums
        t = torch.from_numpy(sums)
        p.dev["sums"].copy_(t.transpose(1, 2) if p.layout == "nhd" else t)
    per = -(-keep // p.page_size)
    assert len(p.free) >= S * per
    new = np.array(p.free[:S * per], np.int32).reshape(S, per)
    kept, count = mq.kv_evict(p.cache, p.pages, p.lens, p.max_len, torch.from_numpy(new).cuda(),
                              keep, sink, recent)
    mq.stream_status()
    kept, count = kept.cpu().numpy(), count.cpu().numpy()
    want = {n: t.copy() for n, t in p.host.items()}
    for s, n in enumerate(p.lens_list):
        assert count[s] == min(n, keep)
        page, slot = kv.place(p.pages_host[s], p.page_size, np.arange(n))
        for h in range(hkv):
            stay = kv.evict(p.host["sums"][page, h, slot], n, keep, sink, recent)
            assert kept[s, h].tolist() == stay + [-1] * (keep - len(stay)), (s, h)
            to, ts = kv.place(new[s], p.page_size, np.arange(len(stay)))
            for name in want:
                want[name][to, h, ts] = p.host[name][page[stay], h, slot[stay]]
    for name in want:
        assert np.array_equal(bits(p.read(name)), bits(want[name])), name
    return kept


def paged(kind, lens, keep, hkv=2, dim=64, page_size=16, layout="hnd", seed=0):
    return Paged(kind, lens, hkv, dim, page_size, layout=layout, sums=True, seed=seed,
                 spare=len(lens) * -(-keep // page_size) + 1)


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_types_and_widths(kind, dim):
    check(paged(kind, [100, 40, 41, 0], 40, dim=dim, seed=dim), 40, 4, 8)


@pytest.mark.parametrize("page_size", [1, 7, 16, 100])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_pages_and_layouts(page_size, layout):
    check(paged("q8_0", [300, 120, 129], 128, hkv=3, page_size=page_size, layout=layout), 128, 2, 30)


@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (64, 64, 0),
                                              (64, 0, 64), (64, 32, 32), (64, 0, 0), (2000, 1, 1)])
def test_budgets(keep, sink, recent):
    check(paged("f16", [1, 2, 65, 500, 1999, 2001], keep, seed=keep), keep, sink, recent)


def test_equal_sums_stay_from_the_lowest_position():
    p = paged("f16", [3000, 777], 500, seed=1)
    rng = np.random.default_rng(2)
    for levels in (1, 2, 5):
        check(p, 500, 3, 40, rng.integers(0, levels, p.host["sums"].shape).astype(np.float32))


def test_special_sums():
    """NaN above infinity, then the numbers, negative ones too, down to minus infinity; -0 is 0."""
    p = paged("f16", [1200], 300, seed=3)
    rng = np.random.default_rng(4)
    w = rng.normal(size=p.host["sums"].shape).astype(np.float32)
    pick = rng.integers(0, 12, w.shape)
    for i, v in enumerate([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45]):
        w[pick == i] = v
    for keep in (20, 150, 300):
        check(p, keep, 0, 0, w)


@pytest.mark.parametrize("S,hkv,n,keep", [(1, 1, 70000, 30000), (1, 4, 131072, 1000), (9, 2, 5000, 4999),
                                          (40, 8, 200, 64)])
def test_sizes(S, hkv, n, keep):
    lens = [n - 3 * i for i in range(S)]
    p = paged("q8_0", lens, keep, hkv=hkv, seed=n)
    w = (np.random.default_rng(5).random(p.host["sums"].shape) ** 8 * 20).astype(np.float32)
    check(p, keep, 4, min(32, keep // 2), w)


def test_a_sequence_with_several_copies_of_one_sum_across_thread_blocks():
    """The tie runs through the whole length: the rows that stay end in its middle."""
    p = paged("f16", [40000], 20000, hkv=1, page_size=64, seed=6)
    w = np.full(p.host["sums"].shape, 2.0, np.float32)
    kept = check(p, 20000, 0, 100, w)
    assert kept[0, 0, 19899] == 19899 and kept[0, 0, 19900] == 39900


@pytest.mark.parametrize("n,hkv", [(4500, 1), (9000, 3), (17000, 2), (40000, 1), (34000, 16),
                                   (270000, 1)])
@pytest.mark.parametrize("shape", ["spread", "close", "levels", "4096 alike", "4097 alike"])
def test_choice_by_one_and_by_several_thread_blocks(n, hkv, shape):
    """The last row that stays lies among few or many whose leading bits are its own."""
    rng = np.random.default_rng(n)
    p = paged("q8_0", [n], 2600, hkv=hkv, page_size=64, seed=n)
    size = p.host["sums"].shape
    if shape == "spread":
        w = rng.random(size) ** 8 * 20
    elif shape == "close":
        w = 1 + rng.random(size) * 1e-3
    elif shape == "levels":
        w = rng.integers(0, 3, size) * 0.5
    else:  # that many rows between 1 and 1.25 of the candidates, 1000 larger, the rest smaller
        w = rng.random(size) * 0.5
        for h in range(hkv):
            at = 4 + rng.permutation(n - 104)[:1000 + int(shape.split()[0])]
            page, slot = kv.place(p.pages_host[0], 64, at)
            w[page[:1000], h, slot[:1000]] = 2 + rng.random(1000)
            w[page[1000:], h, slot[1000:]] = 1 + rng.random(len(at) - 1000) * 0.24
    check(p, 2600, 4, 100, w.astype(np.float32))


def test_bad_lengths_and_pages_are_reported():
    p = paged("f16", [100, 50], 64, seed=7)
    new = torch.tensor(p.free[:8], dtype=torch.int32, device="cuda").view(2, 4)
    lens = torch.tensor([100, 1000], dtype=torch.int32, device="cuda")
    p.pages[1] = p.pages[0]  # clamped to 100, its pages are the first sequence's
    kept, count = mq.kv_evict(p.cache, p.pages, lens, 100, new, 64)
    with pytest.raises(mq.MQError, match="length 1000") as e:
        mq.stream_status()
    assert e.value.name == "MQ_ERR_INDEX"
    assert count.tolist() == [64, 64] and torch.equal(kept[0], kept[1])
    before = p.cache.k.clone()
    bad = new.clone()
    bad[0, 1] = p.cache.n_pages
    mq.kv_evict(p.cache, p.pages, p.lens, 100, bad, 64)
    with pytest.raises(mq.MQError, match="page"):
        mq.stream_status()
    live = ~torch.isnan(before)
    live[new[1].long()] = False
    assert torch.equal(p.cache.k[live], before[live])


def test_refusals_on_the_device():
    p = paged("f16", [100], 64, seed=8)
    new = torch.tensor(p.free[:4], dtype=torch.int32, device="cuda").view(1, 4)
    for kw in (dict(keep=0), dict(keep=64, sink=-1), dict(keep=64, sink=40, recent=25)):
        with pytest.raises(mq.MQError) as e:
            mq.kv_evict(p.cache, p.pages, p.lens, 100, new, **kw)
        assert e.value.name == "MQ_ERR_ARG"
    with pytest.raises(ValueError):
        mq.kv_evict(p.cache, p.pages, p.lens, 100, new, 65)
    with pytest.raises(ValueError):
        mq.kv_evict(p.cache, p.pages, p.lens, 1000, new, 64)
    mq.stream_status()
