"""Value scales that are infinite or NaN beside scales above 1: the other blocks' values keep their sums, over Q8_0 and
Q4_0 rows alike, and queries of every size over Q4_0 rows."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from oracle import kv  # noqa: E402
from tests.kv4_cases import Paged4, attn_bound4  # noqa: E402
from tests.kv_cases import IO, Paged, attn_bound, numpy_of  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


def queries(S, hq, dim, io, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((S, hq, dim), generator=g) * 1.5).to(IO[io])


@pytest.mark.parametrize("kind", ["q8_0", "q4_0"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("size", [1.0, 3.0, 100.0, 10000.0])
@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
def test_beside_scales_that_are_no_numbers(kind, dim, size, what):
    lens = [40, 300]
    p = Paged(kind, lens, 1, dim, 16, seed=4) if kind == "q8_0" else Paged4(lens, 1, dim, 16, seed=4)
    page, slot = kv.place(p.pages_host[1], 16, np.array([50, 210]))
    sc = p.host["v_scale"].astype(np.float32)
    dead = np.isnan(sc)
    sc = np.where(dead, np.nan, np.sign(sc) * (0.5 + np.abs(sc) % 0.5) * size).astype(np.float16)
    sc[page, 0, slot, 1] = what
    p.host["v_scale"] = sc
    t = torch.from_numpy(sc).cuda()
    p.dev["v_scale"] = t
    p.cache = p.wrap()
    q = queries(2, 4, dim, "f32", 5)
    o = mq.attn_decode(p.cache, q.cuda(), p.pages, p.lens, p.max_len).cpu().numpy().astype(np.float64)
    mq.stream_status()
    with np.errstate(invalid="ignore"):
        ref = kv.attn_decode(p.host, 16, numpy_of(q), p.pages_host, p.lens_list, dim ** -0.5)[0]
    finite = {n: np.where(np.isfinite(x), x, 0) for n, x in p.host.items()}
    _, mass, reach, _ = kv.attn_decode(finite, 16, numpy_of(q), p.pages_host, p.lens_list, dim ** -0.5)
    assert np.array_equal(np.isnan(o), np.isnan(ref)) and np.array_equal(np.isinf(o), np.isinf(ref))
    assert (np.sign(o[np.isinf(o)]) == np.sign(ref[np.isinf(ref)])).all()
    fine = np.isfinite(ref)
    assert fine.sum() >= 2 * 4 * dim - 4 * 32
    bound = attn_bound(dim, reach, mass, np.where(fine, ref, 0), "f32")
    if kind == "q4_0":
        p.host.update(finite)
        bound, _ = attn_bound4(p, numpy_of(q), np.where(fine, ref, 0), mass, reach, dim ** -0.5, 0, "f32")
    assert (np.abs(o[fine] - ref[fine]) <= bound[fine]).all()


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -40, 2.0 ** -13, 2.0 ** 10, 2.0 ** 60, 2.0 ** 120])
def test_queries_of_every_size(io, size):
    """The logits' scale undoes the queries' size, where the type holds it."""
    if io == "f16" and not 2.0 ** -14 < size < 2.0 ** 12:
        return
    dim = 128
    p = Paged4([1, 40, 300], 2, dim, 16, seed=6)
    q = (queries(3, 8, dim, "f32", 7) * size).to(IO[io])
    q[:, :, 0] *= 2.0 ** -30 if io != "f16" else 0.5
    scale = dim ** -0.5 / size
    o = mq.attn_decode(p.cache, q.cuda(), p.pages, p.lens, p.max_len, scale=scale)
    mq.stream_status()
    ref, mass, reach, _ = kv.attn_decode(p.host, 16, numpy_of(q), p.pages_host, p.lens_list, scale, 0)
    bound, _ = attn_bound4(p, numpy_of(q), ref, mass, reach, scale, 0, io)
    assert (np.abs(numpy_of(o).astype(np.float64) - ref) <= bound).all()
