"""The paged cache of Q4_0 rows: attention against the 64-bit definition, stored rows bit for bit,
eviction; what no call may read is poisoned."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from oracle import kv  # noqa: E402
from tests.kv4_cases import Paged4, attn_bound4  # noqa: E402
from tests.kv_cases import IO, numpy_of  # noqa: E402


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


def check(p, q, io, dim, window=0, track=False, scale=None, ws=None):
    scale = dim ** -0.5 if scale is None else scale
    o = mq.attn_decode(p.cache, q.cuda(), p.pages, p.lens, p.max_len, scale=scale, window=window, track=track, ws=ws)
    mq.stream_status()
    ref, mass, reach, weights = kv.attn_decode(p.host, p.page_size, numpy_of(q), p.pages_host, p.lens_list, scale,
                                               window)
    err = np.abs(numpy_of(o).astype(np.float64) - ref)
    bound, rel = attn_bound4(p, numpy_of(q), ref, mass, reach, scale, window, io)
    assert (err <= bound).all(), f"worst err/bound {np.max(err / bound):.3g}"
    if track:
        got, want = (x.astype(np.float64) for x in (p.read("sums"), p.host["sums"]))
        slack = np.zeros_like(want)
        group = q.shape[1] // want.shape[1]
        for s, (lo, w) in enumerate(weights):
            page, slot = kv.place(p.pages_host[s], p.page_size, np.arange(lo, lo + w.shape[1]))
            for h in range(w.shape[0] if w.shape[1] else 0):
                want[page, h, slot] += w[h]
                slack[page, h, slot] = (w[h] * np.expm1(rel[s].max()) + np.abs(want[page, h, slot]) * 2.0 ** -22
                                        + group * 1e-37)
        live = ~np.isnan(want)
        assert np.array_equal(live, ~np.isnan(got))
        assert (np.abs(got - want)[live] <= slack[live]).all()
        p.host["sums"] = p.read("sums")
    return o


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200, 511, 513]


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_widths_and_types(dim, io):
    p = Paged4(LENS, 2, dim, 16, seed=dim)
    check(p, queries(len(LENS), 8, dim, io, dim), io, dim)


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (2, 1), (7, 1), (8, 1), (9, 1), (16, 1), (17, 1), (36, 2), (71, 1)])
def test_head_layouts(dim, hq, hkv):
    p = Paged4([130, 5, 0, 67], hkv, dim, 16, seed=hq)
    check(p, queries(4, hq, dim, "f32", hq), "f32", dim)


@pytest.mark.parametrize("page_size", [1, 3, 7, 16, 24, 100, 1000])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("dim", [96, 128])
def test_pages_and_layouts(page_size, layout, dim):
    p = Paged4([1, 130, 999, 24, 0], 3, dim, page_size, layout=layout, seed=page_size)
    check(p, queries(5, 6, dim, "f32", page_size), "f32", dim)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 511, 512, 5000])
def test_sliding_window(window):
    p = Paged4(LENS, 2, 128, 24, seed=window)
    check(p, queries(len(LENS), 4, 128, "f32", window), "f32", 128, window=window)


@pytest.mark.parametrize("dim,hq,hkv", [(128, 28, 4), (96, 12, 12), (64, 14, 2), (256, 20, 1), (192, 4, 4)])
@pytest.mark.parametrize("window", [0, 70])
def test_weight_sums(dim, hq, hkv, window):
    p = Paged4([0, 1, 17, 300, 64, 1025], hkv, dim, 16, sums=True, seed=hq)
    for seed in (1, 2):
        check(p, queries(6, hq, dim, "f32", seed), "f32", dim, window=window, track=True)


@pytest.mark.parametrize("S,n", [(1, 20000), (3, 9000), (1, 50001)])
def test_long_sequences(S, n):
    p = Paged4([n - 37 * i for i in range(S)], 2, 128, 64, seed=n, sums=True)
    check(p, queries(S, 14, 128, "f32", n), "f32", 128, track=True)


def test_many_unlike_sequences():
    rng = np.random.default_rng(5)
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(3000), 150))]
    lens[7] = 9000
    lens[8] = lens[149] = 0
    p = Paged4(lens, 2, 64, 16, seed=6)
    check(p, queries(150, 4, 64, "f32", 7), "f32", 64)


def test_uneven_weights():
    p = Paged4([400, 33], 1, 128, 16, seed=8)
    q = queries(2, 4, 128, "f32", 9)
    check(p, q * 20, "f32", 128)
    check(p, q, "f32", 128, scale=0.0)
    check(p, q, "f32", 128, scale=-0.2)
    check(p, q * 1e-30, "f32", 128)
    check(p, torch.zeros_like(q), "f32", 128)


@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** -5, 1.0, 30.0, 3000.0])
def test_scales_far_from_one(size):
    """Values' scales above 1 (brought below it by a power of two) and far below, zero ones among them."""
    p = Paged4([300, 33, 70], 1, 128, 16, seed=8)
    sc = (np.random.default_rng(3).standard_normal(p.host["v_scale"].shape) * size).astype(np.float16)
    sc[np.isnan(p.host["v_scale"])] = np.nan
    sc[..., 0][:, :, ::3] *= 0
    p.set("v", kv.pack4((p.host["v"] + 8).astype(np.uint8)), sc)
    p.cache = p.wrap()
    check(p, queries(3, 8, 128, "f32", 2), "f32", 128)


def test_scales_that_are_no_numbers():
    """A value's scale that is infinite or NaN makes its block's dims so (NaN where the number is 8:
    0 * inf), and leaves the others alone."""
    p = Paged4([40, 100], 1, 64, 16, seed=4)
    q = queries(2, 4, 64, "f32", 5)
    page, slot = kv.place(p.pages_host[1], 16, np.array([50, 70]))
    sc = p.host["v_scale"].copy()
    sc[page[0], 0, slot[0], 1] = np.inf
    n = (p.host["v"] + 8).astype(np.uint8)
    n[page[0], 0, slot[0], 32:64] = np.arange(32) % 16
    p.set("v", kv.pack4(n), sc)
    p.cache = p.wrap()
    o = mq.attn_decode(p.cache, q.cuda(), p.pages, p.lens, p.max_len).cpu().numpy()
    mq.stream_status()
    with np.errstate(invalid="ignore"):
        ref = kv.attn_decode(p.host, 16, numpy_of(q), p.pages_host, p.lens_list, 64 ** -0.5)[0]
    assert np.array_equal(np.isnan(o), np.isnan(ref)) and np.array_equal(np.isinf(o), np.isinf(ref))
    assert np.array_equal(np.sign(o[np.isinf(o)]), np.sign(ref[np.isinf(ref)]))
    fine = np.isfinite(ref)
    assert fine.sum() == 2 * 4 * 64 - 4 * 32 and np.abs(o[fine] - ref[fine]).max() < 1e-5


def test_bad_pages_and_lengths_are_reported():
    p = Paged4([40, 60], 2, 128, 16, seed=1)
    q = queries(2, 4, 128, "f32", 1).cuda()
    good = mq.attn_decode(p.cache, q, p.pages, p.lens, p.max_len)
    pages = p.pages.clone()
    pages[0, 1] = p.cache.n_pages
    o = mq.attn_decode(p.cache, q, pages, p.lens, p.max_len)
    with pytest.raises(mq.MQError, match="page"):
        mq.stream_status()
    assert torch.equal(o[1], good[1]) and not torch.equal(o[0], good[0])


@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_strided_planes(layout):
    """Layers of one pool, a view of every other page."""
    p = Paged4([77, 300], 2, 96, 16, layout=layout, seed=3)
    q = queries(2, 4, 96, "f32", 6).cuda()
    want = mq.attn_decode(p.cache, q, p.pages, p.lens, p.max_len)
    wide = {n: torch.stack([t, torch.full_like(t, 7)], 1) for n, t in p.dev.items()}
    c = mq.KVCache(mq.Q4_0, *(wide[n][:, 0] for n in ("k", "v", "k_scale", "v_scale")), layout=layout)
    assert torch.equal(mq.attn_decode(c, q, p.pages, p.lens, p.max_len), want)


# ---- stored rows --------------------------------------------------------------------------


def planes(cache, name):
    t = getattr(cache, name)
    return numpy_of(t.transpose(1, 2) if cache.layout == "nhd" else t)


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("pairs,rot", [(False, None), (True, None), (False, 24), (True, 40)])
@pytest.mark.parametrize("T,hq,hkv,layout,io", [(37, 6, 2, "hnd", "f32"), (1, 1, 1, "nhd", "bf16"), (700, 5, 5, "nhd", "f16")])
def test_stored_rows(dim, pairs, rot, T, hq, hkv, layout, io):
    rot = rot or dim
    g = torch.Generator().manual_seed(dim + T)
    ps = 16
    cache = mq.kv_cache(mq.Q4_0, -(-T // ps) + 2, ps, hkv, dim, sums=True, layout=layout)
    for t in (cache.k, cache.v):
        t.fill_(3)
    cache.sums.fill_(5.0)
    slot = torch.randperm(cache.n_pages * ps, generator=g)[:T]
    slot[T // 2] = -1 if T > 1 else slot[0]
    x = (torch.randn((T, (hq + 2 * hkv) * dim), generator=g) * 2).to(IO[io])
    bias = torch.randn(x.shape[1], generator=g)
    table = mq.rope_table(500, [1e4 ** (-2 * i / rot) for i in range(rot // 2)])
    pos = torch.randint(0, 500, (1, T), generator=g, dtype=torch.int32)
    mq.rope_store(cache, mq.Rope(table, pairs=pairs), x.cuda(), pos.cuda(), slot.cuda(), hq, bias=bias.cuda())
    mq.stream_status()
    y = (x.float().numpy() + bias.numpy()).reshape(T, -1, dim)
    y[:, :hq + hkv] = kv.rope(y[:, :hq + hkv], table.cpu().numpy(), pos.numpy().astype(np.int64), [0] * (rot // 2), pairs)
    live = slot.numpy() >= 0
    page, off = slot.numpy()[live] // ps, slot.numpy()[live] % ps
    for name, rows in (("k", y[live, hq:hq + hkv]), ("v", y[live, hq + hkv:])):
        n, d = kv.quantise_rows4(rows)
        want, scales = np.full_like(planes(cache, name), 3), np.zeros_like(planes(cache, name + "_scale"))
        for h in range(hkv):
            want[page, h, off], scales[page, h, off] = kv.pack4(n[:, h]), d[:, h]
        assert np.array_equal(planes(cache, name + "_scale").view(np.uint16), scales.view(np.uint16)), name
        assert np.array_equal(planes(cache, name), want), name
    sums = np.full_like(planes(cache, "sums"), 5.0)
    sums[page, :, off] = 0.0
    assert np.array_equal(planes(cache, "sums"), sums)


def test_zero_blocks_ties_and_large_values():
    cache = mq.kv_cache(mq.Q4_0, 1, 16, 1, 64)
    rope = mq.Rope(mq.rope_table(8, [0.0] * 32))
    x = torch.zeros((6, 3 * 64))
    x[1, 128:134] = torch.tensor([-8.0, 0.5, 1.5, -2.5, 8.0, 7.5])
    x[2, 128] = 3e7
    x[3, 128] = 1e-8
    x[4, 130], x[4, 129] = float("inf"), 5.0
    x[5, 160] = float("nan")
    mq.rope_store(cache, rope, x.cuda(), torch.zeros((1, 6), dtype=torch.int32, device="cuda"),
                  torch.arange(6, device="cuda"), 1)
    mq.stream_status()
    v, sc = cache.v[0, 0].cpu().numpy(), cache.v_scale[0, 0].cpu().numpy()
    want, d = kv.quantise_rows4(x[:5, 128:].numpy())
    assert np.array_equal(sc[:5], d) and np.array_equal(v[:5], kv.pack4(want))
    # the positive one of two alike is the largest: d = -1, and 0.5, 1.5, -2.5, 7.5 by -1 go to the even
    assert sc[1, 0] == -1 and kv.unpack4(v[1:2])[0, :6].tolist() == [15, 8, 6, 10, 0, 0]
    assert sc[2, 0] == -65504 and sc[3, 0] == 0 and sc[4, 0] == -65504 and kv.unpack4(v[4:5])[0, 2] == 0
    assert np.isnan(sc[5, 1]) and sc[5, 0] == 0


# ---- eviction -----------------------------------------------------------------------------


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_eviction_moves_rows(dim, layout):
    p = Paged4([300, 40, 100, 0], 2, dim, 16, layout=layout, sums=True, seed=dim, spare=20)
    keep, sink, recent = 64, 4, 16
    new = torch.tensor(p.free[:16], dtype=torch.int32).view(4, 4)
    before = {n: p.read(n) for n in p.dev}
    kept, lens = mq.kv_evict(p.cache, p.pages, p.lens, p.max_len, new.cuda(), keep, sink=sink, recent=recent)
    mq.stream_status()
    assert lens.tolist() == [64, 40, 64, 0]
    after = {n: p.read(n) for n in p.dev}
    touched = set()
    for s, n in enumerate(p.lens_list):
        for h in range(2):
            page, slot = kv.place(p.pages_host[s], 16, np.arange(n)) if n else (np.zeros(0, int), np.zeros(0, int))
            stay = kv.evict(before["sums"][page, h, slot], n, keep, sink, recent)
            assert kept[s, h].tolist() == stay + [-1] * (keep - len(stay))
            for j, i in enumerate(stay):
                to = (int(new[s, j // 16]), h, j % 16)
                touched.add(to)
                for name in p.dev:
                    a, b = after[name][to], before[name][page[i], h, slot[i]]
                    assert np.array_equal(np.atleast_1d(a).view(np.uint8), np.atleast_1d(b).view(np.uint8)), name
    for name in p.dev:  # and nothing else
        same = before[name].copy()
        for to in touched:
            same[to] = after[name][to]
        assert np.array_equal(same.view(np.uint8), after[name].view(np.uint8))


@pytest.mark.parametrize("S,n,keep", [(3, 5000, 4097), (40, 700, 350)])
def test_eviction_of_many_rows(S, n, keep):
    p = Paged4([n] * S, 3, 96, 16, sums=True, seed=2, spare=S * (-(-keep // 16)))
    new = torch.tensor(p.free[:S * -(-keep // 16)], dtype=torch.int32).view(S, -1)
    kept, _ = mq.kv_evict(p.cache, p.pages, p.lens, p.max_len, new.cuda(), keep, recent=32)
    mq.stream_status()
    for s in (0, S - 1):
        for h in range(3):
            at = kept[s, h].cpu().numpy()
            src, dst = kv.place(p.pages_host[s], 16, at), kv.place(new[s].numpy(), 16, np.arange(keep))
            for name in ("k", "v", "k_scale", "v_scale"):
                x = p.read(name)
                assert np.array_equal(x[dst[0], h, dst[1]].view(np.uint8), x[src[0], h, src[1]].view(np.uint8))


# ---- the binding --------------------------------------------------------------------------


def test_cache_objects():
    c = mq.kv_cache(mq.Q4_0, 2, 8, 3, 96, layout="nhd")
    assert c.k.shape == (2, 8, 3, 48) and c.k_scale.shape == (2, 8, 3, 3) and c.head_dim == 96
    with pytest.raises(ValueError, match="scales"):
        mq.KVCache(mq.Q4_0, c.k, c.v, layout="nhd")
    with pytest.raises(ValueError, match="uint8"):
        mq.KVCache(mq.Q4_0, c.k.view(torch.int8), c.v.view(torch.int8), c.k_scale, c.v_scale, layout="nhd")
    with pytest.raises(ValueError, match="shape"):
        mq.KVCache(mq.Q4_0, c.k, c.v, c.k_scale[..., :2], c.v_scale[..., :2], layout="nhd")
    with pytest.raises(mq.MQError, match="head_dim=32"):
        small = mq.kv_cache(mq.Q4_0, 2, 8, 1, 32)
        mq.attn_decode(small, torch.zeros((1, 1, 32), device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                       torch.ones(1, dtype=torch.int32, device="cuda"), 8)
