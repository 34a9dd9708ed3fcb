"""mq_rope_store with positions on an axis that no pair turns by: the same result as without it."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


@pytest.mark.parametrize("sections", [[20, 12, 0], [32, 0, 0], [0, 32, 0, 0], [16, 0, 16]])
def test_an_empty_section(sections):
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = mq.kv_cache(mq.F16, 2, 16, 2, 64)
    tab = mq.rope_table(100, [1e4 ** (-i / 32) for i in range(32)])
    axis = mq.rope_axes(sections)
    pos = torch.randint(0, 100, (len(sections), 19), dtype=torch.int32, device="cuda", generator=g)
    qkv = torch.randn((19, 8 * 64), device="cuda", generator=g)
    slot = torch.arange(19, device="cuda")
    q = mq.rope_store(cache, mq.Rope(tab, axis, n_axes=len(sections)), qkv, pos, slot, 4)
    k = cache.k.clone()
    used = max(axis) + 1
    q2 = mq.rope_store(cache, mq.Rope(tab, axis), qkv, pos[:used].contiguous(), slot, 4)
    assert torch.equal(q, q2) and torch.equal(k, cache.k)
    mq.stream_status()
