"""mq_norm_rope_store: the heads' norms, the rotation and the stored rows, bit for bit: the norm's
factor is the binary32 nearest to the exact one, the rest as mq_rope_store."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from oracle import kv  # noqa: E402
from tests.kv_cases import IO, numpy_of  # noqa: E402
from tests.test_gpu_rope_store import as_bits, round_to, stored  # noqa: E402

KINDS = {"f16": mq.F16, "bf16": mq.BF16, "q8_0": mq.Q8_0, "q4_0": mq.Q4_0}


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


def normed(x, w, eps):
    """Heads x [T][H][D] normed in binary32, and those whose factor lies within 2^-28 of the middle of
    two binary32 numbers (the kernel's sums and residual hold it to 2^-30; either is right there)."""
    g = kv.head_scale(x, eps)
    f = g.astype(np.float32)
    up, down = np.nextafter(f, np.float32(np.inf)), np.nextafter(f, np.float32(0))
    near = np.minimum(np.abs((f.astype(np.float64) + up) / 2 - g), np.abs((f.astype(np.float64) + down) / 2 - g))
    return (x * f[..., None]) * w, near <= g * 2.0 ** -28


def check(kind, T, hq, hkv, dim, rot=None, axes=1, pairs=False, layout="hnd", io="f32", bias=False, seed=0,
          skip=0.0, eps=1e-6, size=1.0):
    rot, ps = rot or dim, 16
    g = torch.Generator().manual_seed(seed)
    cache = mq.kv_cache(KINDS[kind], -(-T // ps) + 2, ps, hkv, dim, sums=True, layout=layout)
    for t in (cache.k, cache.v):
        t.fill_(3)
    cache.sums.fill_(5.0)
    slot = torch.where(torch.rand(T, generator=g) < skip, -1, torch.randperm(cache.n_pages * ps, generator=g)[:T])
    heads = hq + 2 * hkv
    by = torch.exp(torch.randn((T, heads, 1), generator=g) * 2) * size
    x = (torch.randn((T, heads, dim), generator=g) * by).view(T, heads * dim).to(IO[io])
    b = torch.randn(heads * dim, generator=g) * size if bias else None
    wq, wk = (torch.randn(dim, generator=g) for _ in range(2))
    half = rot // 2
    axis = torch.randint(0, axes, (half,), generator=g).tolist()
    axis[0] = axes - 1
    table = mq.rope_table(500, [1e4 ** (-i / half) for i in range(half)])
    pos = torch.randint(0, 500, (axes, T), generator=g, dtype=torch.int32)
    q = mq.rope_store(cache, mq.Rope(table, axis, pairs), x.cuda(), pos.cuda(), slot.cuda(), hq,
                      bias=None if b is None else b.cuda(), norm=mq.HeadNorm(wq.cuda(), wk.cuda(), eps))
    mq.stream_status()
    y = x.float().numpy()
    if b is not None:
        y = y + b.numpy()
    y = y.reshape(T, heads, dim).copy()
    m = hq + hkv
    w = np.concatenate([np.broadcast_to(wq.numpy(), (hq, dim)), np.broadcast_to(wk.numpy(), (hkv, dim))])
    y[:, :m], tie = normed(y[:, :m], w, np.float32(eps))
    # (binary32 numbers lie 2^-24 to 2^-23 of their size apart: at most 1/8 of the heads on average, and
    # five deviations of that many draws)
    assert tie.mean() <= 1 / 8 + 5 * (7 / 64 / tie.size) ** 0.5
    y[:, :m] = kv.rope(y[:, :m], table.cpu().numpy(), pos.numpy().astype(np.int64), axis, pairs)
    sure = ~tie
    got, want = as_bits(numpy_of(q).reshape(T, hq, dim)), as_bits(round_to(y[:, :hq], io))
    assert np.array_equal(got[sure[:, :hq]], want[sure[:, :hq]])
    # near a tie of the factor: within its last place (and the roundings after it)
    close = np.abs(numpy_of(q).reshape(T, hq, dim).astype(np.float64) - y[:, :hq])
    lim = np.abs(y[:, :hq]).max(-1, keepdims=True) * (2.0 ** -21 + {"f32": 0, "f16": 2.0 ** -10, "bf16": 2.0 ** -7}[io])
    assert (close <= lim + 1e-30).all()
    live = slot.numpy() >= 0
    page, off = slot.numpy()[live] // ps, slot.numpy()[live] % ps
    for name, rows, ok in (("k", y[live, hq:m], sure[live, hq:]), ("v", y[live, m:], np.ones((live.sum(), hkv), bool))):
        have = stored(cache, name)
        touched = np.zeros(have.shape[:3], bool)
        for h in range(hkv):
            touched[page, h, off] = True
            r, mine = rows[:, h], ok[:, h]
            if kind in ("q8_0", "q4_0"):
                quants, d = kv.quantise_rows(r) if kind == "q8_0" else kv.quantise_rows4(r)
                quants = kv.pack4(quants) if kind == "q4_0" else quants
                sc = stored(cache, name + "_scale")[page, h, off]
                assert np.array_equal(as_bits(sc[mine]), as_bits(d[mine])), name
            else:
                quants = round_to(r, kind)
            assert np.array_equal(as_bits(have[page, h, off][mine]), as_bits(quants[mine])), name
        assert (have[~touched] == 3).all()
    sums = np.full_like(stored(cache, "sums"), 5.0)
    sums[page, :, off] = 0.0
    assert np.array_equal(stored(cache, "sums"), sums)


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0", "q4_0"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("pairs", [False, True])
def test_types_and_widths(kind, dim, pairs):
    check(kind, 37, 6, 2, dim, pairs=pairs, axes=3, bias=True, seed=dim)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["f16", "q8_0", "q4_0"])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_activation_types_and_layouts(kind, io, layout):
    check(kind, 50, 4, 4, 128, io=io, layout=layout, bias=io == "bf16", seed=9)


@pytest.mark.parametrize("rot", [8, 24, 64, 104])
@pytest.mark.parametrize("pairs", [False, True])
def test_partial_rotation(rot, pairs):
    for kind in ("f16", "q4_0"):
        check(kind, 21, 5, 1, 128, rot=rot, pairs=pairs, axes=2, seed=rot)


@pytest.mark.parametrize("T", [1, 2, 8, 300, 1111])
@pytest.mark.parametrize("hq,hkv", [(14, 2), (1, 1), (32, 8), (71, 1)])
def test_counts(T, hq, hkv):
    check("q4_0", T, hq, hkv, 64, axes=4, seed=T, bias=True)
    check("q4_0", T, hq, hkv, 96, axes=1, seed=T, skip=0.3)
    check("bf16", T, hq, hkv, 128, axes=1, seed=T, skip=0.3)


@pytest.mark.parametrize("size,eps", [(1e-12, 1e-6), (1e-20, 1e-30), (1e12, 1e-6), (1e19, 1e-6), (2e34, 1e-6),
                                      (1.0, 1e30), (1.0, 1e-30), (1e-3, 1e-6)])
@pytest.mark.parametrize("dim", [64, 96])
def test_sizes_near_the_ends_of_binary32(size, eps, dim):
    """Sums of squares past binary32, heads far below the epsilon."""
    check("bf16", 40, 4, 2, dim, size=size, eps=eps, seed=5)


def test_heads_of_zeros_infinities_and_nan():
    dim = 64
    cache = mq.kv_cache(mq.BF16, 1, 16, 1, dim)
    rope = mq.Rope(mq.rope_table(4, [0.0] * 32))
    x = torch.randn((4, 3 * dim))
    x[0, :] = 0
    x[1, 5] = float("inf")
    x[2, 5] = float("nan")
    one = torch.ones(dim, device="cuda")
    q = mq.rope_store(cache, rope, x.cuda(), torch.zeros((1, 4), dtype=torch.int32, device="cuda"),
                      torch.arange(4, device="cuda"), 1, norm=mq.HeadNorm(one, one)).cpu()[:, 0]
    mq.stream_status()
    assert not q[0].any() and torch.isnan(q[2]).all()
    # (dims 5 and 37 turn together)
    assert torch.isnan(q[1, 5]) and not q[1][[i for i in range(dim) if i not in (5, 37)]].any()
    want = x[3, :dim].double() / (x[3, :dim].double().pow(2).mean() + 1e-6).sqrt()
    assert (q[3] - want).abs().max() < 1e-6


def test_one_token_in_place_and_wide_rows():
    """A single token's queries over its row; rows read from a wider tensor; a captured graph."""
    dim, hq, hkv = 128, 4, 2
    g = torch.Generator().manual_seed(3)
    cache = mq.kv_cache(mq.Q4_0, 4, 16, hkv, dim)
    rope = mq.Rope(mq.rope_table(100, [0.5 ** i for i in range(64)]))
    norm = mq.HeadNorm(torch.randn(dim, generator=g).cuda(), torch.randn(dim, generator=g).cuda())
    x = torch.randn((9, (hq + 2 * hkv) * dim), generator=g).cuda()
    pos, slot = torch.arange(9, dtype=torch.int32, device="cuda"), torch.arange(9, device="cuda")
    want = mq.rope_store(cache, rope, x, pos, slot, hq, norm=norm)
    rows = cache.k.clone(), cache.v.clone()
    wide = torch.randn((9, x.shape[1] + 40), generator=g).cuda()
    wide[:, :x.shape[1]] = x
    assert torch.equal(mq.rope_store(cache, rope, wide[:, :x.shape[1]], pos, slot, hq, norm=norm), want)
    row = x[:1].clone()
    q = mq.rope_store(cache, rope, row, pos[:1], slot[:1], hq, q=row[:, :hq * dim].view(1, hq, dim), norm=norm)
    assert torch.equal(q, want[:1])
    with pytest.raises(mq.MQError, match="overlaps"):
        two = x[:2].clone()
        mq.rope_store(cache, rope, two, pos[:2], slot[:2], hq, q=two.view(-1)[:2 * hq * dim].view(2, hq, dim), norm=norm)
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            mq.rope_store(cache, rope, x, pos, slot, hq, q=out, norm=norm)
    cache.k.zero_(), cache.v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(cache.k, rows[0]) and torch.equal(cache.v, rows[1])
    mq.stream_status()


def test_refusals():
    cache = mq.kv_cache(mq.F16, 1, 16, 1, 64)
    rope = mq.Rope(mq.rope_table(4, [0.0] * 32))
    x, pos, slot = torch.zeros((1, 192), device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="heads of 128"):
        mq.rope_store(cache, rope, x, pos, slot, 1, norm=mq.HeadNorm(torch.ones(128, device="cuda"), torch.ones(128, device="cuda")))
    for bad in (w.half(), w.cpu(), torch.ones((64, 1), device="cuda"), torch.ones(128, device="cuda")[::2], torch.ones(32, device="cuda")):
        with pytest.raises(ValueError):
            mq.HeadNorm(w, bad)
    with pytest.raises(mq.MQError, match="eps"):
        mq.rope_store(cache, rope, x, pos, slot, 1, norm=mq.HeadNorm(w, w, 0.0))
    off = torch.ones(66, device="cuda")[1:65]
    with pytest.raises(mq.MQError) as e:
        mq.rope_store(cache, rope, x, pos, slot, 1, norm=mq.HeadNorm(off, w))
    assert e.value.name == "MQ_ERR_ALIGN"
