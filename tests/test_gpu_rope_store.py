"""mq_rope_store: the rotated queries and the stored rows against the definition, bit for bit in
binary32 and within rounding of 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from oracle import kv  # noqa: E402
from tests.kv_cases import IO, KINDS, numpy_of  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


def make(kind, T, hq, hkv, dim, rot, axes, page_size, layout, io, bias, seed, skip=0.0):
    g = torch.Generator().manual_seed(seed)
    n_pages = -(-T // page_size) + 2
    cache = mq.kv_cache(KINDS[kind], n_pages, page_size, hkv, dim, sums=True, layout=layout)
    for t in (cache.k, cache.v):
        t.fill_(3)
    cache.sums.fill_(5.0)
    order = torch.randperm(n_pages * page_size, generator=g)[:T]
    slot = torch.where(torch.rand(T, generator=g) < skip, -1, order)
    width = (hq + 2 * hkv) * dim
    x = (torch.randn((T, width), generator=g) * 2).to(IO[io])
    b = torch.randn(width, generator=g) if bias else None
    half = rot // 2
    axis = torch.randint(0, axes, (half,), generator=g).tolist()
    axis[0] = axes - 1
    max_pos = 500
    table = mq.rope_table(max_pos, [1e4 ** (-i / half) for i in range(half)])
    pos = torch.randint(0, max_pos, (axes, T), generator=g, dtype=torch.int32)
    return cache, slot, x, b, axis, table, pos


def stored(cache, name):
    t = getattr(cache, name)
    return numpy_of(t.transpose(1, 2) if cache.layout == "nhd" else t)


def as_bits(a):
    return np.ascontiguousarray(a).view({2: np.uint16, 4: np.uint32, 1: np.uint8}[a.dtype.itemsize])


def round_to(x, io):
    """f32 values rounded to a type and back, as numpy (f16) or torch (bf16) round."""
    return numpy_of(torch.from_numpy(np.ascontiguousarray(x)).to(IO[io]))


def check(kind, T, hq, hkv, dim, rot=None, axes=1, pairs=False, page_size=16, layout="hnd",
          io="f32", bias=False, seed=0, skip=0.0):
    rot = rot or dim
    cache, slot, x, b, axis, table, pos = make(kind, T, hq, hkv, dim, rot, axes, page_size, layout,
                                               io, bias, seed, skip)
    rope = mq.Rope(table, axis, pairs)
    q = mq.rope_store(cache, rope, x.cuda(), pos.cuda(), slot.cuda(), hq,
                      bias=None if b is None else b.cuda())
    mq.stream_status()
    xf = x.float().numpy()
    if b is not None:
        xf = xf + b.numpy()
    xf = xf.reshape(T, -1, dim)
    tab, p = table.cpu().numpy(), pos.numpy().astype(np.int64)
    y = xf.copy()
    y[:, :hq + hkv] = kv.rope(xf[:, :hq + hkv], tab, p, axis, pairs)
    exact = kv.rope(xf[:, :hq + hkv].astype(np.float64), tab.astype(np.float64), p, axis, pairs)
    size = np.abs(xf[:, :hq + hkv]).max() * 2
    # three roundings of values below `size`
    assert np.abs(y[:, :hq + hkv] - exact).max() <= 3 * 2.0 ** -24 * size * 2
    assert np.array_equal(as_bits(numpy_of(q)), as_bits(round_to(y[:, :hq], io)))
    live = slot.numpy() >= 0
    page, off = slot.numpy()[live] // page_size, slot.numpy()[live] % page_size
    for name, rows in (("k", y[live, hq:hq + hkv]), ("v", y[live, hq + hkv:])):
        want = np.full_like(stored(cache, name), 3)
        if kind == "q8_0":
            quants, d = kv.quantise_rows(rows)
            scales = np.zeros_like(stored(cache, name + "_scale"))
            for h in range(hkv):
                want[page, h, off], scales[page, h, off] = quants[:, h], d[:, h]
            assert np.array_equal(as_bits(stored(cache, name + "_scale")), as_bits(scales)), name
        else:
            for h in range(hkv):
                want[page, h, off] = round_to(rows[:, h], kind)
        assert np.array_equal(as_bits(stored(cache, name)), as_bits(want)), name
    sums = np.full_like(stored(cache, "sums"), 5.0)
    sums[page, :, off] = 0.0
    assert np.array_equal(stored(cache, "sums"), sums)


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("pairs", [False, True])
def test_types_and_widths(kind, dim, pairs):
    check(kind, 37, 6, 2, dim, pairs=pairs, axes=3, bias=True, seed=dim)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["f16", "q8_0"])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_activation_types_and_layouts(kind, io, layout):
    check(kind, 50, 4, 4, 128, io=io, layout=layout, page_size=7, bias=io == "bf16", seed=9)


@pytest.mark.parametrize("rot", [8, 16, 24, 48, 64, 104, 120])
@pytest.mark.parametrize("pairs", [False, True])
def test_partial_rotation(rot, pairs):
    """Rotated parts that end inside a 32-element block, or whose halves do."""
    for kind in ("f16", "q8_0"):
        check(kind, 21, 5, 1, 128, rot=rot, pairs=pairs, axes=2, seed=rot)


@pytest.mark.parametrize("T", [1, 2, 8, 300, 1111])
@pytest.mark.parametrize("hq,hkv", [(14, 2), (1, 1), (32, 8), (71, 1)])
def test_counts(T, hq, hkv):
    check("f16", T, hq, hkv, 64, axes=4, seed=T, bias=True)
    check("q8_0", T, hq, hkv, 96, axes=1, seed=T, skip=0.3)


def test_rows_are_read_from_a_wider_tensor():
    cache, slot, x, b, axis, table, pos = make("f16", 9, 4, 2, 64, 64, 1, 16, "hnd", "f32", False, 3)
    wide = torch.randn((9, x.shape[1] + 40))
    wide[:, :x.shape[1]] = x
    rope = mq.Rope(table, axis)
    q = mq.rope_store(cache, rope, x.cuda(), pos.cuda(), slot.cuda(), 4)
    q2 = mq.rope_store(cache, rope, wide.cuda()[:, :x.shape[1]], pos.cuda(), slot.cuda(), 4)
    assert torch.equal(q, q2)
    with pytest.raises(mq.MQError) as e:  # rows of 513 floats are not 16-byte aligned
        mq.rope_store(cache, rope, torch.zeros((9, 513), device="cuda")[:, :512], pos.cuda(),
                      slot.cuda(), 4)
    assert e.value.name == "MQ_ERR_ALIGN"


def test_zero_blocks_ties_and_large_values():
    """Rows of zeros have scale 0; ties round to the even quant; a scale past f16's range is held
    at 65504."""
    cache = mq.kv_cache(mq.Q8_0, 1, 16, 1, 64)
    rope = mq.Rope(mq.rope_table(4, [0.0] * 32))
    x = torch.zeros((4, 3 * 64))
    x[1, 128:132] = torch.tensor([127.0, 0.5, 1.5, -2.5])
    x[2, 128] = 3e7
    x[3, 128] = 1e-7
    mq.rope_store(cache, rope, x.cuda(), torch.zeros((1, 4), dtype=torch.int32, device="cuda"),
                  torch.arange(4, device="cuda"), 1)
    v, sc = cache.v[0, 0].cpu(), cache.v_scale[0, 0].cpu()
    want, d = kv.quantise_rows(x[:, 128:].numpy())
    assert np.array_equal(v[:4].numpy(), want) and np.array_equal(sc[:4].numpy(), d)
    assert v[1, :4].tolist() == [127, 0, 2, -2] and sc[2, 0] == 65504 and sc[3, 0] == 0
    mq.stream_status()


def test_bad_positions_and_slots_are_reported():
    cache, slot, x, b, axis, table, pos = make("f16", 6, 2, 1, 64, 64, 2, 16, "hnd", "f32", False, 5)
    rope = mq.Rope(table, axis)
    good = mq.rope_store(cache, rope, x.cuda(), pos.cuda(), slot.cuda(), 2)
    mq.stream_status()
    for bad in (-1, 500, 1 << 30):
        p2 = pos.clone()
        p2[1, 3] = bad
        q = mq.rope_store(cache, rope, x.cuda(), p2.cuda(), slot.cuda(), 2)
        with pytest.raises(mq.MQError, match=f"position {bad}") as e:
            mq.stream_status()
        assert e.value.name == "MQ_ERR_INDEX"
        assert not q[3].any() and torch.equal(q[:3], good[:3]) and torch.equal(q[4:], good[4:])
    before = cache.k.clone()
    s2 = slot.clone()
    s2[2] = cache.n_pages * cache.page_size
    q = mq.rope_store(cache, rope, x.cuda(), pos.cuda(), s2.cuda(), 2)
    with pytest.raises(mq.MQError, match="slot"):
        mq.stream_status()
    mq.stream_status()
    assert torch.equal(q, good) and torch.equal(cache.k, before)
    # nothing to do
    mq.rope_store(cache, rope, x[:0].cuda(), pos[:, :0].contiguous().cuda(), slot[:0].cuda(), 2)
    mq.stream_status()
