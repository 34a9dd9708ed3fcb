"""Attention over Q4_0 rows keeps what two f16 parts of a weight hold, whatever the activations' type and however
small the values' scales: bounds without a term for weights of fewer bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from oracle import kv  # noqa: E402
from tests.kv4_cases import Paged4, attn_bound4  # noqa: E402
from tests.kv_cases import IO, numpy_of, tiny  # noqa: E402

BITS = {"f32": 24, "f16": 11, "bf16": 8}


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


def check(p, q, io, scale):
    o = mq.attn_decode(p.cache, q.cuda(), p.pages, p.lens, p.max_len, scale=scale)
    mq.stream_status()
    ref, mass, reach, _ = kv.attn_decode(p.host, p.page_size, numpy_of(q), p.pages_host, p.lens_list, scale, 0)
    _, rel = attn_bound4(p, numpy_of(q), ref, mass, reach, scale, 0, io)
    # What f16 holds of small weights: a weight (2^15 for the largest) and its product with a scale d below 1 end in three
    # roundings to steps of 2^-24, half a step each: a key with a number of at most 8 loses 8 * 3 * 2^-25 of
    # 2^15 in units of `unit`, a power of two up to twice the largest scale (2^-15 at least: smaller scales are
    # brought up by 2^15).
    unit = max(2.0 ** -15, 2 * float(np.nanmax(np.abs(p.host["v_scale"].astype(np.float64)))))
    floor = np.array([24 * n * 2.0 ** -40 * unit for n in p.lens_list])[:, None, None]
    near = floor + np.expm1(rel)[..., None] * mass
    # the rounding to the output's type: half a step of the binade that the value lies in
    step = np.exp2(np.floor(np.log2(np.abs(ref) + near + 1e-300))) * 2.0 ** -BITS[io]
    err = np.abs(numpy_of(o).astype(np.float64) - ref)
    bound = near + step + tiny(io)
    assert (err <= bound).all(), f"worst err/bound {np.max(err / bound):.3g}, {np.mean(err > bound):.3g} of all"


def queries(S, hq, dim, io, seed, size=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((S, hq, dim), generator=g) * size).to(IO[io])


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_rounded_once(dim, io):
    """Few keys, so that the errors of their weights do not cancel: the output's rounding is the only one of its
    size."""
    lens = [1, 2, 2, 3, 3, 5, 9, 17, 33] * 4
    p = Paged4(lens, 2, dim, 16, seed=dim)
    check(p, queries(len(lens), 14, dim, io, dim), io, dim ** -0.5)


@pytest.mark.parametrize("size", [0.7, 2.0 ** -4, 2.0 ** -9, 2.0 ** -14, 2.0 ** -20])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_light_keys_beside_a_heavy_one(dim, size):
    """The heavy key's value is zero: what is left are weights of 2^-16 to 2^-36 of the largest."""
    S, hq = 2, 14
    p = Paged4([2, 3], 1, dim, 16, seed=1)
    kn, vn = ((p.host[x] + 8).astype(np.uint8) for x in ("k", "v"))
    ks, vs = (p.host[x + "_scale"].copy() for x in ("k", "v"))
    for s in range(S):
        page, slot = kv.place(p.pages_host[s], 16, np.arange(p.lens_list[s]))
        kn[page, 0, slot] = 8                       # logits of zero ...
        kn[page[0], 0, slot[0]] = 15                # ... but for the first key's
        ks[page, 0, slot] = 0.125
        vn[page[0], 0, slot[0]] = 8
        vs[page, 0, slot] = size
    p.set("k", kv.pack4(kn), ks)
    p.set("v", kv.pack4(vn), vs)
    p.cache = p.wrap()
    # logit = scale * sum q k = q dim 0.875 scale: (16 + 20 i / hq) ln 2
    want = torch.tensor([(16 + 20 * i / hq) * math.log(2) for i in range(hq)])
    q = (want / (dim * 0.875 * dim ** -0.5))[None, :, None].expand(S, hq, dim).contiguous()
    check(p, q, "f32", dim ** -0.5)


@pytest.mark.parametrize("size", [2.0 ** -8, 2.0 ** -12, 2.0 ** -16, 2.0 ** -20])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_small_scales(size, dim):
    p = Paged4([300, 33, 70, 5], 1, dim, 16, seed=8)
    sc = (np.random.default_rng(3).standard_normal(p.host["v_scale"].shape) * size).astype(np.float16)
    sc[np.isnan(p.host["v_scale"])] = np.nan
    p.set("v", kv.pack4((p.host["v"] + 8).astype(np.uint8)), sc)
    p.cache = p.wrap()
    check(p, queries(4, 8, dim, "f32", 2), "f32", dim ** -0.5)


def test_tiles_of_unlike_scales():
    """Small scales, then large ones, then small ones: each tile's power of two is its own."""
    p = Paged4([2000], 1, 128, 16, seed=9)
    rng = np.random.default_rng(4)
    sc = rng.standard_normal(p.host["v_scale"].shape)
    page, slot = kv.place(p.pages_host[0], 16, np.arange(2000))
    size = np.exp2(rng.integers(-20, 12, 2000 // 50).repeat(50).astype(np.float64))
    sc[page, 0, slot] *= size[:, None]
    sc = sc.astype(np.float16)
    sc[np.isnan(p.host["v_scale"])] = np.nan
    p.set("v", kv.pack4((p.host["v"] + 8).astype(np.uint8)), sc)
    p.cache = p.wrap()
    check(p, queries(1, 28, 128, "f32", 3), "f32", 128 ** -0.5)
