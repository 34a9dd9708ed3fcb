"""The value that an index error names, for indexes past 32 bits."""
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


@pytest.mark.parametrize("slot", [16, (1 << 31) - 1, 1 << 31, (1 << 32) + 5, (1 << 62) + 3])
def test_a_slot_past_the_cache_is_named(slot):
    cache = mq.kv_cache(mq.F16, 1, 16, 1, 64)
    rope = mq.Rope(mq.rope_table(4, [0.0] * 32))
    for _ in range(2):  # (and the words are clear after a report)
        mq.rope_store(cache, rope, torch.ones((1, 3 * 64), device="cuda"),
                      torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                      torch.tensor([slot], device="cuda"), 1)
        with pytest.raises(mq.MQError, match=f"slot {slot} is outside") as e:
            mq.stream_status()
        assert e.value.name == "MQ_ERR_INDEX"
        mq.stream_status()
    assert not cache.k.any()
