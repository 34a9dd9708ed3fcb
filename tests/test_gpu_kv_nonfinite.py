"""mq_attn_decode on infinities and NaN in rows that are read, and on queries near the ends of
binary32, against the 64-bit definition: which outputs are infinite, which are NaN, and the values
of all others."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from oracle import kv  # noqa: E402
from tests.kv_cases import Paged, attn_bound  # noqa: E402

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


def put(p, name, s, head, pos, dim, value):
    """One element (of a Q8_0 cache: the scale of its block) of a live row, on both sides."""
    page, slot = kv.place(p.pages_host[s], p.page_size, pos)
    if p.kind == "q8_0":
        name, dim = name + "_scale", dim // 32
    p.host[name][page, head, slot, dim] = value
    at = (int(page), head, int(slot)) if p.layout == "hnd" else (int(page), int(slot), head)
    p.dev[name][at][dim] = value


def queries(S, hq, dim, seed):
    return torch.randn((S, hq, dim), generator=torch.Generator().manual_seed(seed))


def check(p, q, window=0, scale=None, track=False):
    """Infinities and NaN where the definition has them, the rest within the bound of the finite
    elements (their part of a product with an infinity has no size)."""
    dim = q.shape[-1]
    scale = dim ** -0.5 if scale is None else scale
    o = mq.attn_decode(p.cache, q.cuda(), p.pages, p.lens, p.max_len, scale=scale, window=window, track=track)
    mq.stream_status()
    o = o.cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        ref, _, _, weights = kv.attn_decode(p.host, p.page_size, q.numpy(), p.pages_host, p.lens_list, scale, window)
    finite = {n: np.where(np.isfinite(t), t, 0) for n, t in p.host.items()}
    _, mass, reach, _ = kv.attn_decode(finite, p.page_size, q.numpy(), p.pages_host, p.lens_list, scale, window)
    assert np.array_equal(np.isnan(o), np.isnan(ref)), (np.isnan(o).sum(), np.isnan(ref).sum())
    assert np.array_equal(np.isinf(o), np.isinf(ref)) and (np.sign(o[np.isinf(o)]) == np.sign(ref[np.isinf(o)])).all()
    fine = np.isfinite(ref)
    bound = attn_bound(dim, reach, mass, np.where(fine, ref, 0), "f32")
    assert (np.abs(o[fine] - ref[fine]) <= bound[fine]).all()
    return o, ref, weights


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (14, 2), (12, 1), (17, 1)])
def test_values(kind, dim, hq, hkv):
    """An infinite value makes its dim infinite, two of unlike signs or a NaN make it NaN; the other
    dims, heads and sequences are as without."""
    p = Paged(kind, [300, 1, 40, 129], hkv, dim, 24, seed=dim)
    last = hkv - 1
    put(p, "v", 0, 0, 17, 1, INF)
    put(p, "v", 0, 0, 290, 40, -INF)
    put(p, "v", 2, last, 39, dim - 1, INF)
    put(p, "v", 2, last, 3, dim - 1, -INF)
    put(p, "v", 3, last, 128, 33, NAN)
    put(p, "v", 3, last, 0, dim - 2, INF)
    o, ref, _ = check(p, queries(4, hq, dim, hq))
    assert np.isnan(ref).any() and not np.isfinite(ref).all() and np.isfinite(ref).any()
    if kind != "q8_0":
        assert np.isinf(ref).any()


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
def test_the_heaviest_key_has_the_infinite_value(kind):
    """(its weight is a power of two: what is left of it for further parts is zero)"""
    for at in (0, 33, 99):
        p = Paged(kind, [100], 1, 128, 16, seed=1)
        q = queries(1, 3, 128, 2)
        page, slot = kv.place(p.pages_host[0], 16, at)
        if kind != "q8_0":
            k = (q[0, 0] * 3).to(p.dev["k"].dtype)
            p.dev["k"][int(page), 0, int(slot)] = k.cuda()
            p.host["k"][page, 0, slot] = k.float().numpy()
        put(p, "v", 0, 0, at, 5, INF)
        check(p, q)
    p = Paged(kind, [1], 1, 128, 16, seed=3)
    put(p, "v", 0, 0, 0, 100, -INF)
    check(p, queries(1, 1, 128, 4))


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("page_size,layout", [(16, "hnd"), (7, "nhd")])
def test_values_of_long_sequences(kind, page_size, layout):
    """One piece of a split length has them; and a window that ends behind or before them."""
    p = Paged(kind, [20001, 700], 2, 128, page_size, layout=layout, seed=5)
    put(p, "v", 0, 1, 12345, 70, INF)
    put(p, "v", 0, 0, 20000, 0, -INF)
    put(p, "v", 1, 1, 100, 3, INF)
    q = queries(2, 6, 128, 6)
    check(p, q)
    check(p, q, window=20001 - 12345)
    check(p, q, window=20001 - 12346)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("group", [1, 7, 12, 17])
def test_keys(kind, dim, group):
    """A key whose logit is minus infinity weighs nothing; plus infinity or NaN makes the head NaN.
    The sums of the weights take the same."""
    p = Paged(kind, [200, 65, 1100], 2, dim, 16, sums=True, seed=group)
    q = queries(3, 2 * group, dim, dim)
    q[0, :, 10] = q[0, :, 10].abs() + 0.1   # of either sign by head below
    q[0, 1::2, 10] *= -1
    q[1, :, 3] = q[1, :, 3].abs() + 0.1
    q[2, :, dim - 1] = -q[2, :, dim - 1].abs() - 0.1
    put(p, "k", 0, 0, 150, 10, INF)
    put(p, "k", 1, 1, 64, 3, -INF)
    put(p, "k", 1, 1, 2, 3, -INF)
    put(p, "k", 2, 0, 1000, dim - 1, INF)
    put(p, "k", 2, 1, 4, 0, NAN)
    before = p.host["sums"].copy()
    o, ref, weights = check(p, q, track=True)
    assert np.isnan(ref[0, :group:2]).all() and np.isfinite(ref[0, 1:group:2]).all()
    assert np.isfinite(ref[1]).all() and np.isfinite(ref[2, :group]).all() and np.isnan(ref[2, group:]).all()
    sums = p.read("sums").astype(np.float64)
    for s, (lo, w) in enumerate(weights):
        page, slot = kv.place(p.pages_host[s], 16, np.arange(w.shape[1]))
        for h in range(2):
            want = before[page, h, slot] + w[h]
            got = sums[page, h, slot]
            assert np.array_equal(np.isnan(got), np.isnan(want)), (s, h)
            fine = ~np.isnan(want)  # (2^-12: well above what these logits' errors make of a weight)
            assert (np.abs(got - want)[fine] <= (w[h] * 2.0 ** -12 + np.abs(want) * 2.0 ** -22)[fine]).all()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_no_key_weighs_anything(kind):
    """All logits minus infinity: as without keys, zeros."""
    p = Paged(kind, [40, 40], 1, 64, 16, seed=7)
    q = queries(2, 2, 64, 8)
    q[0, :, 0] = -1.0
    for i in range(40):
        put(p, "k", 0, 0, i, 0, INF)
    o = mq.attn_decode(p.cache, q.cuda(), p.pages, p.lens, p.max_len)
    assert not o[0].any() and o[1].all()
    mq.stream_status()


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("power", [127, 126, 120, 116, 100, -100, -116, -120, -125])
def test_queries_near_the_ends_of_binary32(kind, power):
    """Scaled queries with the inverse scale are the same attention."""
    p = Paged(kind, [200, 33], 1, 128, 16, seed=9)
    q = queries(2, 3, 128, 10)
    q /= q.abs().max(-1, keepdim=True).values * 1.01  # (largest element 0.99)
    check(p, q * 2.0 ** power, scale=2.0 ** -power)


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
def test_one_key_outweighs_all(kind):
    """Logits of 2^90 and more apart: the largest takes all, and o is its value (2^-17: the bound's
    part that does not come from the logits)."""
    p = Paged(kind, [200], 1, 128, 16, seed=11)
    q = queries(1, 3, 128, 12)
    page, slot = kv.place(p.pages_host[0], 16, np.arange(200))
    k, v = (kv.values(p.host, n)[page, 0, slot] for n in ("k", "v"))
    for power, scale in ((100, 0.1), (110, 0.1), (110, -0.1), (118, 0.01), (0, 2.0 ** 110), (126, 2.0 ** -20)):
        x = q * 2.0 ** power / 8
        o = mq.attn_decode(p.cache, x.cuda(), p.pages, p.lens, p.max_len, scale=scale)[0].cpu().numpy()
        want = v[(scale * (x[0].double().numpy() @ k.T)).argmax(-1)]
        assert (np.abs(o - want) <= 2.0 ** -17 * np.abs(want)).all(), (power, scale)
    mq.stream_status()
