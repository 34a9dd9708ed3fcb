"""The example's layer at the end of its rotation table."""
import pytest

import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from gguf_block_quantized_q4_gb300.examples import decode_layer  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


def test_a_step_past_the_last_position_is_refused():
    K, rows = 256, 4 * 64
    layer = decode_layer.DecodeLayer(
        mq.register_weight(mq.Q4_K, synth.weights(synth.Q4_K, rows, K, 1), rows, K),
        mq.register_weight(mq.Q8_0, synth.weights(synth.Q8_0, 128, 128, 2), 128, 128),
        2, 2, 1, 64, limit=8, keep=4, sink=1, recent=2, max_pos=20)
    x = torch.randn((2, K), device="cuda")
    for _ in range(20):
        layer.step(x)
    mq.stream_status()
    held = list(layer.held)
    with pytest.raises(ValueError, match="position 20"):
        layer.step(x)
    assert layer.held == held and layer.seen == 20
