"""mq_kv_evict with the new lengths written over the old ones."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from tests.test_gpu_kv_evict import paged  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


@pytest.mark.parametrize("lens,hkv,keep", [([300], 4, 64), ([100000], 2, 1000), ([9000, 40, 0, 6001], 3, 500),
                                           ([2000 - 13 * i for i in range(60)], 8, 32)])
def test_lengths_updated_in_place(lens, hkv, keep):
    """One and several thread blocks a head, and more heads than run at once: a block that comes late
    must still choose by the old length."""
    p = paged("q8_0", lens, keep, hkv=hkv, page_size=64, seed=hkv)
    per = -(-keep // 64)
    new = torch.tensor(p.free[:len(lens) * per], dtype=torch.int32, device="cuda").view(len(lens), per)
    kept, count = mq.kv_evict(p.cache, p.pages, p.lens, p.max_len, new, keep, 4, 16)
    assert count.tolist() == [min(n, keep) for n in lens]
    sums, k = p.cache.sums.clone(), p.cache.k.clone()
    for _ in range(20):
        n = p.lens.clone()
        again, same = mq.kv_evict(p.cache, p.pages, n, p.max_len, new, keep, 4, 16, new_lens=n)
        assert same is n and torch.equal(n, count) and torch.equal(again, kept)
    mq.stream_status()
    assert torch.equal(p.cache.k, k) and torch.equal(p.cache.sums.nan_to_num(-1), sums.nan_to_num(-1))
